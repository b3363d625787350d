"""Plain 64-bit forms of the 4-bit weight and mixture-of-experts operators
with the spread that fp32 rounding leaves them, for long sums, where the
worst case of every rounding (op_util) is larger than the results.

The model.  A rounding is off by at most u = 2^-24 of what is rounded, on
its own account: the errors of a sum of n terms add as squares.  What is
rounded is a partial sum, and terms x w with x of random sign (the tests')
make it a random walk: its square is about the sum of the terms' squares
passed so far, never far above the sum V of all.  A sum of n terms then has a
variance of at most n u^2 V; 4 n u^2 V is taken, since the largest partial sum of a
walk is at most twice its end on average (Doob).  With 4-bit weights the terms
of a group are x (16 + q) and x (16 + z), 2 G of them, then scaled and added to
the other groups.  A result passes if it is within 8 standard deviations and
half a step of its type, element by element, and if the whole is within 4:
the model is generous, so that neither is a matter of chance, and a lost
block, an exchanged matrix or a wrong offset is far outside both.
"""
from __future__ import annotations

import torch

from op_util import DT, HALF, LIP, U

EACH, WHOLE = 8.0, 4.0


def parts(w, N, K):
    """(q, z, s), fp64 [N, K], of a weight's arrays, on their device."""
    codes, scales, zeros = w
    n = torch.arange(N, device=codes.device)[:, None]
    k = torch.arange(K, device=codes.device)[None, :]
    i, kq, j = k % 128 // 32, k % 32 // 8, k % 8
    byte = kq * 256 + n % 16 * 16 + i * 4 + 2 * (j % 2) + j // 4
    q = codes[n // 16, k // 128, byte].to(torch.int32) >> (4 * (j // 2 % 2)) & 15
    at = (n // 16, k // 128, n % 16, k % 128 // (128 // scales.shape[-1]))
    z = torch.full((N, K), 8.0, dtype=torch.float64, device=codes.device) if zeros is None else (zeros[at] & 15).double()
    return q.double(), z, scales[at].double()


def product(x, w, N, K):
    """(value, variance) of x @ W^T before its rounding: x fp64 [M, K], w a
    tensor [N, K] or a weight's arrays."""
    u2, x2 = U * U, x * x
    if torch.is_tensor(w):
        d = w.double()
        return x @ d.t().contiguous(), 4 * (K + 32) * u2 * (x2 @ (d * d).t().contiguous())
    q, z, s = parts(w, N, K)
    G = 128 // w[1].shape[-1]
    d, s2 = (q - z) * s, s * s
    v = x @ d.t().contiguous()
    inside = x2 @ (s2 * ((16 + q) ** 2 + (16 + z) ** 2)).t().contiguous()
    across = x2 @ (d * d).t().contiguous()
    return v, 4 * u2 * ((2 * G + 8) * inside + (K // G + 32) * across + 4 * v * v)


def activation(v, name):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return 0.5 * v * (1 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v ** 3)))


def layer(x, ids, weights, gate_up, down, I, act, out):
    """(y, variance) of a layer of experts before y's rounding: x a tensor
    [T, H] of its type, ids a list of lists, weights fp64 [T, k];
    gate_up(e, 0 or 1) and down(e) an expert's matrices."""
    T, H = x.shape
    bits = {torch.float16: 22, torch.bfloat16: 24 if out == "f32" else 16}[x.dtype]
    least = 2.0 ** -25 if x.dtype is torch.float16 else 0.0
    xd = x.double()
    y, var = torch.zeros_like(xd), torch.zeros_like(xd)
    for e in sorted({i for row in ids for i in row if i >= 0}):
        at = [(t, j) for t, row in enumerate(ids) for j, i in enumerate(row) if i == e]
        t, j = (torch.tensor(c, device=x.device) for c in zip(*at))
        g, vg = product(xd[t], gate_up(e, 0), I, H)
        u, vu = product(xd[t], gate_up(e, 1), I, H)
        a = activation(g, act)
        va = LIP ** 2 * vg + (16 * U * g) ** 2
        h = a * u
        vh = u * u * va + a * a * vu + (2 * U * h) ** 2 + (2.0 ** -bits * h) ** 2 + least ** 2
        w = down(e)
        d, vd = product(h, w, H, I)
        if not torch.is_tensor(w):
            q, z, s = parts(w, H, I)
            w = (q - z) * s
        wd = w.double()
        vd = vd + vh @ (wd * wd).t().contiguous()
        p = weights[t, j][:, None]
        y.index_add_(0, t, p * d)
        var.index_add_(0, t, p * p * (vd + (20 * U * d) ** 2))
    return y, var


def check(got, value, var, out, label=""):
    g = got.detach().to(value.device).double()
    assert g.shape == value.shape and torch.isfinite(g).all(), label
    rel, least = HALF[out]
    sd = var.sqrt()
    step = torch.clamp((value.abs() + EACH * sd) * rel, min=least)
    off = (g - value).abs()
    whole = WHOLE * float(var.sum().sqrt()) + float(step.norm())
    assert float(off.norm()) <= whole, "%s: %.3g of %.3g off as a whole, at most %.3g" % (
        label, float(off.norm()), float(value.norm()), whole)
    bad = off > EACH * sd + step
    assert not bad.any(), "%s: %d of %d outside 8 standard deviations, the worst by a factor of %.3g" % (
        label, int(bad.sum()), bad.numel(), float((off / (EACH * sd + step)).max()))
