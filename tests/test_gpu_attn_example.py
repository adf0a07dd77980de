"""The example stack of Falcon and softmax-attention layers: stepped tokens
against one prompt call.  The cache rounds keys and values to 4 bits (2^-5 on
average at most); through two attention layers beside the residual stream and
the Falcon layers that stays below 2^-4 of the result."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("lengths,steps", [((70, 1, 33), 20), ((128,), 3), ((5, 200), 40)])
def test_steps_follow_the_prompt(lengths, steps):
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(lengths, steps) < 2.0 ** -4
