"""The losses beside autograd: their results never require grad, and a function
of the two calls passes their gradients on (loss_util has the bounds)."""
import pytest
import torch

import dense_gemm_tiled_amd as tg
import loss_util as lu
from test_gpu_cross_entropy import case

pytestmark = pytest.mark.gpu


class HeadLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, targets):
        loss, lse = tg.cross_entropy(x, w, targets)
        ctx.save_for_backward(x, w, targets, lse)
        return loss

    @staticmethod
    def backward(ctx, grad):
        x, w, targets, lse = ctx.saved_tensors
        return (*tg.cross_entropy_backward(x, w, targets, lse, grad, torch.empty_like(x), torch.empty_like(w)), None)


def test_results_never_require_grad():
    x, w, targets, g = case(20, 100, 64, "f32")
    logits = torch.randn(20, 8, device="cuda", generator=g)
    for t in (x, w, logits):
        t.requires_grad_()
    ids, weights = tg.moe_route(logits, 2)
    results = [*tg.cross_entropy(x, w, targets), weights, *tg.moe_balance(logits, ids)]
    assert not any(t.requires_grad for t in results)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [9, 200])
def test_a_function_of_the_two_calls(dtype, T):
    """The mean (an expanded grad) and a weighted sum in one backward pass."""
    x, w, targets, g = case(T, 300, 64, dtype)
    weight = torch.rand(T, device="cuda", generator=g)
    x.requires_grad_(), w.requires_grad_()
    (HeadLoss.apply(x, w, targets).mean()).backward()
    means = x.grad.clone(), w.grad.clone()
    x.grad = w.grad = None
    (HeadLoss.apply(x, w, targets) * weight).sum().backward()
    lse = tg.cross_entropy(x, w, targets)[1]
    for got, grad in ((means, torch.full((T,), 1.0 / T, device="cuda")), ((x.grad, w.grad), weight)):
        want = lu.grads64(x.detach(), w.detach(), targets, lse, grad, 1.0, dtype, dtype, dtype)
        lu.check(got[0], *want["dx"], dtype, "dx")
        lu.check(got[1], *want["dw"], dtype, "dw")
