"""Probabilities of a router around fp32's smallest ordinary number (loss_util
has the bounds)."""
import pytest
import torch

import dense_gemm_tiled_amd as tg
import loss_util as lu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [12, 13, 60, 256, 509])
@pytest.mark.parametrize("renormalize", [True, False])
def test_what_is_below_2_to_the_minus_126_counts_as_0(E, renormalize):
    """Logits of 0 to -110 below the largest: what is above 2^-126 (-87.3) has its
    gradient, what is below 2^-128 (-88.7) may have 0, off by at most its own
    share, and finite rows stay finite."""
    T, k = 220, 2
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = -torch.arange(T, device="cuda")[:, None] * 0.5 * torch.rand(T, E, device="cuda", generator=g)
    logits[:, E // 2] = 0.0
    ids, _ = tg.moe_route(logits, k)
    dw, slope = torch.randn(T, k, device="cuda", generator=g), torch.randn(E, device="cuda", generator=g)
    loss, counts, _ = tg.moe_balance(logits, ids)
    want, n, _, off, _ = lu.balance64(logits, ids, 1.0)
    assert torch.equal(counts.long(), n) and abs(float(loss.double() - want)) <= off + 2.0 ** -24 * abs(float(want))
    d = tg.moe_route_backward(logits, ids, dw, torch.empty_like(logits), renormalize=renormalize, slope=slope,
                              dloss=torch.ones((), device="cuda"))
    value, off = lu.route_grad64(logits, ids, dw, renormalize, 1.0, slope, torch.ones((), device="cuda"))
    # (a share of p below 2^-126, its own or in the places' sums, times what it is multiplied by)
    least = 2.0 ** -126 * 4 * float(slope.abs().max() + dw.abs().sum(1).max())
    assert torch.isfinite(d).all() and ((d.double() - value).abs() <= off + 2.0 ** -24 * value.abs() + least).all()
    far = logits < -88.8
    far.scatter_(1, ids.long(), False)
    assert far.any() and (d[far] == 0).all()
