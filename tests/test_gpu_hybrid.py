"""The example that runs the recurrent layer, the cache and the attention together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "hybrid_step.py")


@pytest.mark.parametrize("prompts, steps", [((700, 1, 129, 64), 8), ((63,), 3)])
def test_decoded_equals_prefilled(prompts, steps):
    spec = importlib.util.spec_from_file_location("hybrid_step", _path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    diff, _, _ = example.run(prompts, steps)
    assert diff <= example.BOUND
