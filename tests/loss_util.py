"""Plain 64-bit forms of the losses of a training step (the cross entropy of a
linear layer, a router's balance loss) and of their gradients, with the
spread that the kernels' roundings leave them.

The products.  A product is a sum of H terms in fp32: as in op_spread, its
errors add as squares, a variance of at most 4 (H + 32) u^2 sum x^2 w^2, u =
2^-24.  What is made of it afterwards moves by as much as its slope says:
lse by sum_v p_v dl_v, p_v by p_v times (dl_v - dlse).

The sums.  lse adds V positive numbers, in chains of at most V / 64 + 64 (32 in
a lane or 8 in a row's share, then over lanes, waves and shares): a relative
gamma_n.  An exponential is off by 2^-22 (its own last places and its
argument's, which where it is large is multiplied by a small exponential), the
factors that join shares by as much again: 64 u in all.  The logarithm and the
last sum are off by u of their results: 4 u (|lse| + |l|).

The gradient.  G is rounded to the inputs' type: half a step of it for a
result of that type, 2^-24 (three bf16 numbers), 2^-22 (two f16) or 2^-24 (f32)
for an fp32 result, and f16 has nothing below 2^-25 where the largest grad is
at least 2^14.  Each error moves the result by its own weight, never more than
sum_v |dG| |w|; as independent errors, uniform inside half a step, they leave a
variance of a third of the squares' sum.  The second product's own fp32 sums
count as above, the result's rounding by half a step of its type.

The router.  An exponential's relative error is u times its argument's size
and 4 u of its own, twice (the sum's too): p is off by (64 + 4 |l - max|) u of
itself, and what is made of p by a few u of each of its terms.
"""
from __future__ import annotations

import torch

from op_util import HALF, U

EACH, WHOLE = 8.0, 4.0
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAME = {v: k for k, v in DT.items()}


def gamma(n):
    return n * U / (1.0 - n * U)


def counted(targets, V):
    return (targets >= 0) & (targets < V)


def products(x, w, scale):
    """(l, standard deviation of its error), fp64 [T, V]."""
    xd, wd = x.double(), w.double()
    l = scale * torch.matmul(xd, wd.t().contiguous())
    sd = 2 * U * (x.size(1) + 32) ** 0.5 * abs(scale) * torch.matmul(xd * xd, (wd * wd).t().contiguous()).sqrt()
    return l, sd + U * l.abs()


def loss64(x, w, targets, scale=1.0):
    """loss, lse and how far each may be off, fp64 [T]."""
    V = w.size(0)
    l, sd = products(x, w, scale)
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    off = (p * EACH * sd).sum(1) + gamma(V / 64 + 64) + 64 * U + 4 * U * lse.abs()
    c = counted(targets, V)
    at = torch.where(c, targets, torch.zeros_like(targets)).long()[:, None]
    lt, st = l.gather(1, at)[:, 0], sd.gather(1, at)[:, 0]
    zero = torch.zeros_like(lse)
    loss = torch.where(c, lse - lt, zero)
    return loss, lse, torch.where(c, off + EACH * st + 4 * U * lt.abs(), zero), off


def grads64(x, w, targets, lse, grad, scale, dtype, out_dx, out_dw, dw_old=None, beta=0.0):
    """{"dx": (value, bound of each error, variance), "dw": ..} in fp64, the
    results' own rounding not included."""
    V = w.size(0)
    c = counted(targets, V)
    g = torch.where(c, grad.double().expand(x.size(0)), torch.zeros((), dtype=torch.float64, device=x.device))
    live = g != 0
    # (what a token that adds nothing holds is of no account)
    xd = torch.where(live[:, None], x.double(), torch.zeros((), dtype=torch.float64, device=x.device))
    wd = w.double()
    l, sd = products(xd, wd, scale)
    lse = torch.where(live, lse.double(), torch.zeros_like(g))[:, None]
    p = torch.where(live[:, None], torch.exp(l - lse), torch.zeros_like(l))
    q = p.clone()
    t = torch.nonzero(live)[:, 0]
    q[t, targets[t].long()] -= 1
    G = g[:, None] * q
    soft = g.abs()[:, None] * p * (EACH * sd + 16 * U + 8 * U * (l.abs() + lse.abs()))
    top = float(g.abs().max()) if g.numel() else 0.0
    out = {}
    for name, kind in (("dx", out_dx), ("dw", out_dw)):
        if kind is None:
            continue
        if kind == "f32" and dtype != "f32":
            rel = 2.0 ** -24 if dtype == "bf16" else 2.0 ** -22
        else:
            rel = HALF[dtype][0]
        least = 2.0 ** -39 * top if dtype == "f16" else 0.0
        dG = rel * G.abs() + soft + least * (G != 0)
        vG = (rel * G) ** 2 / 3 + (soft / EACH) ** 2 + (least * (G != 0)) ** 2
        if name == "dx":
            a, b, n = (G, dG, vG), wd, V
        else:
            a, b, n = (G.t().contiguous(), dG.t().contiguous(), vG.t().contiguous()), xd, x.size(0)
        value = scale * torch.matmul(a[0], b)
        sums = 4 * (n + 64) * U * U * scale * scale * torch.matmul(a[0] ** 2, b * b)
        each = abs(scale) * torch.matmul(a[1], b.abs()) + EACH * sums.sqrt()
        var = scale * scale * torch.matmul(a[2], b * b) + sums
        if name == "dw" and beta != 0.0:
            value = value + beta * dw_old.double()
            each = each + 4 * U * (beta * dw_old.double()).abs() * (3 if kind == "f32" else 1)
            var = var + (8 * U * beta * dw_old.double()) ** 2
        out[name] = (value, each, var)
    return out


def check(got, value, each, var, kind, label=""):
    """A result of type `kind` against its value."""
    g = got.detach().double()
    assert g.shape == value.shape and torch.isfinite(g).all(), label
    rel, least = HALF[kind]
    step = torch.clamp((value.abs() + each) * rel, min=least)
    off = (g - value).abs()
    bad = off > each + step
    assert not bad.any(), "%s: %d of %d are further off than they may be, the worst by a factor of %.3g" % (
        label, int(bad.sum()), bad.numel(), float((off / (each + step)).max()))
    if var is not None:
        whole = WHOLE * float(var.sum().sqrt()) + float(step.norm())
        assert float(off.norm()) <= whole, "%s: %.3g of %.3g off as a whole, at most %.3g" % (
            label, float(off.norm()), float(value.norm()), whole)


# ------------------------------------------------------------------ router
def router64(logits, ids):
    """(l with -inf for what has no part, p, counts, alive), fp64."""
    E = logits.size(1)
    big = torch.finfo(torch.float32).max
    l = logits.double()
    l = torch.where(torch.isnan(l), -float("inf"), l).clamp(max=big)
    inside = (ids >= 0) & (ids < E)
    alive = inside.any(1)
    m = l.max(1, keepdim=True).values.clamp(min=-big)
    e = torch.where(l > -float("inf"), torch.exp(l - m), 0.0)
    p = torch.where(alive[:, None], e / e.sum(1, keepdim=True).clamp(min=1e-300), 0.0)
    counts = torch.zeros(E, dtype=torch.int64, device=l.device)
    for j in range(ids.size(1)):
        counts += torch.bincount(ids[inside[:, j], j].long(), minlength=E)
    return l, p, counts, alive


def balance64(logits, ids, coef):
    """loss, counts, slope and the errors that loss and slope may have."""
    E = logits.size(1)
    l, p, counts, alive = router64(logits, ids)
    n, total = int(alive.sum()), int(counts.sum())
    if total == 0:
        z = torch.zeros(E, dtype=torch.float64, device=l.device)
        return z[0], counts, z, 0.0, z
    S = p.sum(0)
    m = l.max(1, keepdim=True).values
    spread = torch.where(p > 0, (m - l).clamp(max=200), 0.0)
    pe = (p * (64 + 4 * spread) * U).sum(0) + gamma(logits.size(0) / 256 + 64) * S
    f = coef * E * counts.double() / total / n
    slope = coef * (E * counts - total).double() / total / n
    return (f * S).sum(), counts, slope, float((f.abs() * pe).sum() + 4 * U * (f * S).sum().abs()), 4 * U * slope.abs()


def route_grad64(logits, ids, dweights, renormalize, scale, slope, dloss):
    """dlogits and the error each may have, fp64."""
    T, E = logits.shape
    l, p, _, alive = router64(logits, ids)
    m = l.max(1, keepdim=True).values
    size = torch.where(p > 0, (m - l).clamp(max=200), 0.0)
    rel = (64 + 4 * size) * U
    d, off = torch.zeros_like(p), torch.zeros_like(p)
    rows = torch.arange(T, device=l.device)
    if dweights is not None:
        at = torch.where((ids >= 0) & (ids < E), ids, 0).long()
        lc = torch.where((ids >= 0) & (ids < E), l.gather(1, at), -float("inf"))
        part = lc > -float("inf")
        dw = torch.where(part, dweights.double(), 0.0)
        if renormalize:
            top = lc.max(1, keepdim=True).values.clamp(min=-3.5e38)
            e = torch.where(part, torch.exp(lc - top), 0.0)
            q = e / e.sum(1, keepdim=True).clamp(min=1e-300)
            s = torch.where(part, (top - lc).clamp(max=200), 0.0)
        else:
            q = p.gather(1, at) * part
            s = torch.where(part, (m - lc).clamp(max=200), 0.0)
        qrel = (80 + 4 * s) * U
        wd = scale * q * dw
        total = wd.sum(1, keepdim=True)
        te = (wd.abs() * qrel).sum(1, keepdim=True) + 20 * U * wd.abs().sum(1, keepdim=True)
        for j in range(ids.size(1)):
            own = wd[:, j] - (q[:, j] * total[:, 0] if renormalize else 0.0)
            oe = (wd[:, j] * qrel[:, j]).abs()
            if renormalize:
                oe = oe + q[:, j] * te[:, 0] + (q[:, j] * qrel[:, j] * total[:, 0]).abs()
            ok = part[:, j]
            d.index_put_((rows[ok], at[ok, j]), own[ok], accumulate=True)
            off.index_put_((rows[ok], at[ok, j]), oe[ok] + 4 * U * own[ok].abs(), accumulate=True)
        if not renormalize:
            d -= p * total
            off += p * te + p * rel * total.abs()
    if slope is not None:
        sl, dl = slope.double(), dloss.double()
        mean = (p * sl).sum(1, keepdim=True)
        me = (p * rel * sl.abs()).sum(1, keepdim=True) + 20 * U * (p * sl.abs()).sum(1, keepdim=True)
        d += dl * p * (sl - mean)
        off += dl.abs() * (p * rel * (sl - mean).abs() + p * me + 4 * U * p * (sl.abs() + mean.abs()))
    off = off + 4 * U * d.abs() + 8 * U * off
    dead = ~alive[:, None]
    return d.masked_fill(dead, 0.0), off.masked_fill(dead, 0.0)
