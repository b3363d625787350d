"""A step of training as a user would run it: tokens routed over experts, a
head over a vocabulary, both losses and all gradients of head and router in
the framework, against autograd in 64 bits."""
import pytest
import torch

import dense_gemm_tiled_amd as tg
import loss_util as lu

pytestmark = pytest.mark.gpu


def test_step():
    T, H, E, k, V, coef = 200, 128, 16, 2, 1000, 0.1
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, router = rnd(T, H), rnd(E, H) / H ** 0.5
    experts, head = rnd(E, H, H) / H ** 0.5, rnd(V, H) * (2.0 / H ** 0.5)
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    targets[::9] = -100
    n = int(lu.counted(targets, V).sum())

    # the framework, fp32: forward
    logits = torch.empty(T, E, device="cuda")
    tg.gemm(x, router, logits, transpose_b=True)
    ids, weights = tg.moe_route(logits, k)
    balance, counts, slope = tg.moe_balance(logits, ids, coef=coef)
    each = torch.stack([experts[ids[:, j].long()] @ x[:, :, None] for j in range(k)], 1)[..., 0]      # [T, k, H]
    y = x + (weights[..., None] * each).sum(1)
    loss, lse = tg.cross_entropy(y, head, targets)
    total = loss.sum() / n + balance
    # and backward
    dy, dhead = torch.empty_like(y), torch.empty_like(head)
    tg.cross_entropy_backward(y, head, targets, lse, torch.full((), 1.0 / n, device="cuda"), dy, dhead)
    dweights = (each * dy[:, None, :]).sum(-1).contiguous()
    dlogits = torch.empty_like(logits)
    tg.moe_route_backward(logits, ids, dweights, dlogits, slope=slope, dloss=torch.ones((), device="cuda"))
    drouter = torch.empty_like(router)
    tg.gemm(dlogits, x, drouter, transpose_a=True)

    # 64 bits, autograd
    xd, rd, hd = x.double(), router.double().requires_grad_(), head.double().requires_grad_()
    ld = xd @ rd.t()
    ld.retain_grad()
    chosen = ld.gather(1, ids.long())
    wd = torch.softmax(chosen, 1)
    ed = each.double()
    yd = xd + (wd[..., None] * ed).sum(1)
    logp = torch.log_softmax(yd @ hd.t(), 1)
    at = targets.clamp(min=0)[:, None]
    ce = -(logp.gather(1, at)[:, 0] * lu.counted(targets, V)).sum() / n
    share = torch.bincount(ids.flatten().long(), minlength=E).double() / (T * k)
    want = ce + coef * E * (share * torch.softmax(ld, 1).mean(0)).sum()
    want.backward()
    assert torch.equal(counts.long(), torch.bincount(ids.flatten().long(), minlength=E))
    # fp32 sums of at most 1000 terms, two products deep: 2^-16 of the whole is
    # 256 roundings, each of them at most 2^-24 of it
    for name, got, ref in (("loss", total, want.detach()), ("dhead", dhead, hd.grad), ("dlogits", dlogits, ld.grad),
                           ("drouter", drouter, rd.grad)):
        off = float((got.double() - ref).norm() / ref.norm())
        assert off <= 2.0 ** -16, (name, off)
