"""The training example: it runs in both dtypes, and its fp32 gradients follow the
differences of its loss.  A central difference of step h is off by h^2 / 6 of the
loss's third derivative along the direction (2^-8 of the slope is allowed for it,
directions of unit length) and by two roundings of the loss, whose terms carry some
2^-18 of fp32 noise through the layers, over h."""

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m():
    spec = importlib.util.spec_from_file_location("hybrid_training", os.path.join(ROOT, "examples", "hybrid_training.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps_run(m, dtype):
    losses = m.main(B=2, T=70, steps=2, dtype=dtype)
    assert len(losses) == 2 and all(math.isfinite(x) for x in losses)


def test_gradients_follow_differences(m):
    g = torch.Generator().manual_seed(4)
    x, target = (torch.randn((2, 70, m.WIDTH), generator=g).cuda() for _ in range(2))
    stack = m.Stack(0, 70, torch.float32)
    m.loss_of(stack, x, target).backward()
    h = 2.0 ** -5
    for name, w in stack.named_parameters():
        u = torch.randn(w.shape, generator=g).cuda()
        u = u / u.norm() + w.grad / w.grad.norm()  # along the gradient too: a slope that stands out of the noise
        u = u / u.norm()
        with torch.no_grad():
            w.add_(h * u)
            hi = m.loss_of(stack, x, target).item()
            w.sub_(2 * h * u)
            lo = m.loss_of(stack, x, target).item()
            w.add_(h * u)
        slope = (w.grad.double() * u).sum().item()
        assert abs((hi - lo) / (2 * h) - slope) <= 2.0 ** -8 * abs(slope) + 2.0 ** -18 * max(hi, lo) / h, name
