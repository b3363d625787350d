"""Gradients whose sizes are near the ends of fp32's range (loss_util has the
bounds)."""
import pytest
import torch

import loss_util as lu
from test_gpu_cross_entropy import backward, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [9, 70])
@pytest.mark.parametrize("size", [3e-34, 1e35])
def test_grads_near_the_ends_of_fp32(size, T, dtype):
    """Results in f32, which hold them: words' weights and tokens' numbers are
    about 0.3 and 1, so sums of T <= 70 stay below 1e37.  (3e-34 is above 2^-112:
    the largest grad becomes 2^14 or more, and f16 keeps 2^-39 of it.)"""
    x, w, targets, g = case(T, 300, 64, dtype)
    grad = (torch.rand(T, device="cuda", generator=g) + 0.5) * size
    assert float(grad.max()) >= 2.0 ** -112
    backward(x, w, targets, grad, dx="f32", dw="f32")

