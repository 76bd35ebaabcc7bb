"""Refusals of the key/value cache calls on the CPU, beyond shapes and addresses."""
import math

import pytest

import kda_state_chunked_gb300 as kda
from kda_state_chunked_gb300 import build as kbuild
from test_kv_host import attn_args


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("T", [0, 3])
def test_attention_refuses_a_scale_that_is_no_number(scale, T):
    pool, args = attn_args(scale=scale, T=T)
    assert kda.lib().kda_attn_paged(*args) == kda.KDA_EINVAL


def test_attention_takes_any_finite_scale():
    for scale in (0.0, -0.1, 1e-40, 3e38):
        pool, args = attn_args(scale=scale, T=0)
        assert kda.lib().kda_attn_paged(*args) == kda.KDA_OK
