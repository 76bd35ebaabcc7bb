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


# ------------------------------------------------------------------ the binding
def tokens():
    torch = pytest.importorskip("torch")
    pool = kda.Pool(kda.kda_kv_page_bytes(2, 64, kda.KDA_KV_I8, 32), 4)
    i = torch.zeros(2, dtype=torch.int32)
    return torch, pool, torch.zeros(3, 2, 64), i


def test_binding_refuses_tables_of_another_type():
    torch, pool, x, i = tokens()
    for bad in (torch.zeros(8, 32, dtype=torch.int32), torch.zeros(8, 32, dtype=torch.float64),
                torch.zeros(8, 32, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="cos_sin must be float32"):
            kda.kda_kv_append(pool, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, None, x, x, bad, None, i)
    for bad in (torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="lse must be float32"):
            kda.kda_attn_paged(pool, 2, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, x, x, i, i, lse=bad)


def test_binding_refuses_a_status_of_another_type():
    torch, pool, x, i = tokens()
    for bad in (torch.zeros(1), torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(ValueError, match="status"):
            kda.kda_kv_append(pool, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, None, x, x, None, None, bad)
        with pytest.raises(ValueError, match="status"):
            kda.kda_kv_gather(pool, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), x, x, bad)
        with pytest.raises(ValueError, match="status"):
            kda.kda_attn_paged(pool, 2, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, x, x, i, bad)


def test_binding_refuses_tensors_of_another_gpu():
    class On:
        """As much of a tensor as the address checks look at."""
        shape = (3, 2, 64)

        def __init__(self, gpu):
            self.gpu = gpu

        def get_device(self):
            return self.gpu

        def is_contiguous(self):
            return True

        def stride(self):
            return (128, 64, 1)

        def data_ptr(self):
            return 4096

    assert kda._address(On(0), 0) == 4096 and kda._rows(On(1), 2, 64, 1) == (4096, 128)
    for at, gpu in ((1, 0), (0, 1), (-1, 0)):
        with pytest.raises(ValueError):
            kda._address(On(at), gpu)
        with pytest.raises(ValueError):
            kda._rows(On(at), 2, 64, gpu)
