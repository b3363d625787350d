"""The losses' operators where offsets pass 32 bits: a weight and its gradient of
more than 4 GiB, rows far apart (loss_util has the bounds)."""
import pytest
import torch

import dense_gemm_tiled_amd as tg
import loss_util as lu

pytestmark = pytest.mark.gpu


def lse64(x, w, scale, step=65536):
    """(lse, its bound) in 64 bits, a part of the words at a time."""
    parts, offs = [], []
    for v in range(0, w.size(0), step):
        l, sd = lu.products(x, w[v:v + step], scale)
        parts.append(torch.logsumexp(l, 1))
        offs.append((torch.exp(l - parts[-1][:, None]) * lu.EACH * sd).sum(1))
    parts, offs = torch.stack(parts, 1), torch.stack(offs, 1)
    lse = torch.logsumexp(parts, 1)
    V = w.size(0)
    off = (torch.exp(parts - lse[:, None]) * offs).sum(1) + lu.gamma(V / 64 + 64) + 64 * lu.U
    return lse, off + 4 * lu.U * lse.abs()


@pytest.mark.parametrize("T,V,H,dtype", [(3, 600001, 4096, "bf16"), (40, 600001, 4096, "f16"), (300, 600001, 4096, "bf16"),
                                         (140, 600001, 4095, "bf16"), (5, 300001, 4096, "f32"), (70, 300001, 4099, "f32")])
def test_weight_past_4_gib(T, V, H, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    w = torch.empty(V, H, dtype=lu.DT[dtype], device="cuda").normal_(0.0, 2.0 / H ** 0.5, generator=g)
    x = torch.randn(T, H, device="cuda", generator=g).to(lu.DT[dtype])
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    targets[0], targets[1] = V - 1, V - 2
    loss, lse = tg.cross_entropy(x, w, targets)
    want, off = lse64(x, w, 1.0)
    lu.check(lse, want, off, None, "f32", "lse")
    lt, st = lu.products(x, w[targets], 1.0)
    lt, st = lt.diagonal(), st.diagonal()
    lu.check(loss, want - lt, off + lu.EACH * st + 4 * lu.U * lt.abs(), None, "f32", "loss")
    grad = torch.rand(T, device="cuda", generator=g) + 0.1
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    tg.cross_entropy_backward(x, w, targets, lse, grad, dx, dw)
    # in 64 bits a part of the words at a time; dw of the first and the last
    rel, least = lu.HALF[dtype][0], 2.0 ** -39 * float(grad.max()) if dtype == "f16" else 0.0
    g64, lse_, xd = grad.double()[:, None], lse.double()[:, None], x.double()
    total = each = square = 0.0
    for v in range(0, V, 65536):
        wd = w[v:v + 65536].double()
        l, sd = lu.products(x, w[v:v + 65536], 1.0)
        p = torch.exp(l - lse_)
        G = g64 * p
        at = torch.nonzero((targets >= v) & (targets < v + wd.size(0)))[:, 0]
        G[at, targets[at] - v] -= grad.double()[at]
        soft = g64 * p * (lu.EACH * sd + 16 * lu.U + 8 * lu.U * (l.abs() + lse_.abs()))
        dG = rel * G.abs() + soft + least
        total = total + torch.matmul(G, wd)
        each = each + torch.matmul(dG, wd.abs())
        square = square + torch.matmul(G * G, wd * wd)
        if v == 0 or v + wd.size(0) == V:
            Gt, dGt = G.t().contiguous(), dG.t().contiguous()
            sums = 2 * lu.U * (T + 64) ** 0.5 * torch.matmul(Gt * Gt, xd * xd).sqrt()
            lu.check(dw[v:v + 65536], torch.matmul(Gt, xd), torch.matmul(dGt, xd.abs()) + lu.EACH * sums, None, dtype,
                     "dw from word %d" % v)
    lu.check(dx, total, each + lu.EACH * 2 * lu.U * (V + 64) ** 0.5 * square.sqrt(), None, dtype, "dx")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_router_rows_far_apart(dtype):
    """2^31 elements and more between the first row and the last."""
    T, E, k, ld = 3001, 60, 4, 800000
    g = torch.Generator(device="cuda").manual_seed(1)
    flat = torch.zeros((T - 1) * ld + E, dtype=lu.DT[dtype], device="cuda")
    logits = flat.as_strided((T, E), (ld, 1))
    logits.copy_(torch.randn(T, E, device="cuda", generator=g))
    ids = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    near = logits.contiguous()
    dweights = torch.randn(T, k, device="cuda", generator=g)
    a, b = tg.moe_balance(logits, ids), tg.moe_balance(near, ids)
    for one, other in zip(a, b):
        assert torch.equal(one, other)
    dfar = torch.zeros_like(flat).as_strided((T, E), (ld, 1))
    dnear = torch.empty_like(near)
    dloss = torch.ones((), device="cuda")
    tg.moe_route_backward(logits, ids, dweights, dfar, renormalize=True, scale=1.0, slope=a[2], dloss=dloss)
    tg.moe_route_backward(near, ids, dweights, dnear, renormalize=True, scale=1.0, slope=a[2], dloss=dloss)
    assert torch.equal(dfar.contiguous(), dnear)
