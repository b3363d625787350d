"""Plain 64-bit forms of the 4-bit weight and mixture-of-experts operators,
on the CPU, with the error bounds the tests hold the kernels to.

Bounds.  u = 2^-24 is half a step of fp32.  A sum of n fp32 terms in any
order is within gamma_n = n u / (1 - n u) of the sum of the terms' sizes.  A
product with 4-bit weights sums x (16 + q) and x (16 + z) per group (2 G
terms), multiplies by s and adds the groups, so its n is 2 K + 2 groups plus
a handful and its terms' sizes are |x| |s| ((16 + q) + (16 + z)).  Rounding
to a 16-bit type adds half a step of it: 2^-8 (bf16) or 2^-11 (f16) of the
value, never less than half its smallest number.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a step relative to the value, and half the smallest number above zero
HALF = {"f32": (2.0 ** -24, 2.0 ** -150), "f16": (2.0 ** -11, 2.0 ** -25),
        "bf16": (2.0 ** -8, 2.0 ** -134)}
LIP = 1.13          # the largest slope of silu (1.0998) and gelu_tanh (1.1290)


def gamma(n):
    return n * U / (1.0 - n * U)


def half_step(v, dtype):
    rel, least = HALF[dtype]
    return np.maximum(rel * np.abs(v), least)


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ the format
def block_position(k):
    """(byte inside a row's 64, shift) of column k of a block."""
    i, kq, j = k // 32, k % 32 // 8, k % 8
    return kq * 256 + i * 4 + 2 * (j & 1) + j // 4, 4 * (j // 2 % 2)


def unpack(codes, N, K):
    """Codes [NB, KB, 1024] as whole numbers [N, K]."""
    c = codes.cpu().numpy()
    out = np.zeros((N, K), np.int64)
    rows = np.arange(N)
    for k in range(K):
        byte, shift = block_position(k % 128)
        out[:, k] = c[rows // 16, k // 128, byte + 16 * (rows % 16)] >> shift & 15
    return out


def per_column(t, N, K, group):
    """Scales or zeros [NB, KB, 16, 128/G] as fp64 [N, K]."""
    a = f64(t)
    n, k = np.arange(N)[:, None], np.arange(K)[None, :]
    return a[n // 16, k // 128, n % 16, k % 128 // group]


def w4_parts(w, N, K):
    """(q, z, s), all fp64 [N, K]."""
    codes, scales, zeros = w
    group = 128 // scales.shape[-1]
    z = np.full((N, K), 8.0) if zeros is None else per_column(zeros, N, K, group)
    return unpack(codes, N, K).astype(np.float64), z, per_column(scales, N, K, group)


def w4_values(w, N, K):
    q, z, s = w4_parts(w, N, K)
    return (q - z) * s


def w4_random(gen, lead, N, K, dtype, group, zeros, device, pad=True):
    """Random weights; with pad, everything past N and K that the format
    stores is set to what would show if it were used (code 15, scale NaN)."""
    nb, kb = -(-N // 16), -(-K // 128)
    q = torch.randint(0, 16, (*lead, nb * 16, kb * 128), generator=gen)
    gp = 128 // group
    s = (torch.rand(*lead, nb, kb, 16, gp, generator=gen) + 0.5) / math.sqrt(K) * 0.3
    s = s * torch.where(torch.rand(s.shape, generator=gen) < 0.5, -1.0, 1.0)
    z = torch.randint(0, 16, s.shape, generator=gen).to(torch.uint8) if zeros else None
    if pad:
        q[..., N:, :] = 15
        q[..., K:] = 15
        n = torch.arange(nb * 16).reshape(nb, 1, 16, 1)
        k = (torch.arange(kb * gp) * group).reshape(1, kb, 1, gp)
        s = torch.where((n >= N) | (k >= K), float("nan"), s)
    codes = np.zeros((int(np.prod(lead, dtype=np.int64)), nb, kb, 1024), np.uint8)
    qn = q.reshape(-1, nb, 16, kb, 128).numpy().astype(np.uint8)
    for k in range(128):
        byte, shift = block_position(k)
        for r in range(16):
            codes[:, :, :, byte + 16 * r] |= qn[:, :, r, :, k] << shift
    codes = torch.from_numpy(codes.reshape(*lead, nb, kb, 1024))
    return (codes.to(device), s.to(DT[dtype]).to(device), None if z is None else z.to(device))


def quantize_ref(w, group, zeros, dtype):
    """(codes [N, K], zero points and scales [N, groups]) of w [N, K] (a CPU
    tensor), by the documented formulas; quotients in fp64, which tells every
    tie of a 24-bit number over an 11-bit one apart."""
    N, K = w.shape
    q, zs, ss = [], [], []
    for k0 in range(0, K, group):
        v = w[:, k0:k0 + group].float()
        bad = ~torch.isfinite(v).all(1, keepdim=True)
        hi, lo = v.amax(1, keepdim=True), v.amin(1, keepdim=True)
        top = torch.finfo(DT[dtype]).max
        if zeros:
            hi, lo = hi.clamp(min=0), lo.clamp(max=0)
            s32 = (hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32)
        else:
            s32 = torch.where(-lo > hi, lo, hi) / -8
        s = s32.clamp(-top, top).to(DT[dtype])
        s = torch.where(bad, torch.tensor(float("nan"), dtype=s.dtype), s)
        d = s.double()
        none = ~(d.abs() > 0)
        dd = torch.where(none, 1.0, d)
        if zeros:
            z = torch.where(none, 0.0, torch.round(-lo.double() / dd).clamp(0, 15))
            c = torch.where(none, z, (torch.round(v.double() / dd) + z).clamp(0, 15))
        else:
            z = torch.full_like(d, 8.0)
            c = torch.where(none, z, torch.round(v.double() / dd).clamp(-8, 7) + 8)
        q.append(c), zs.append(z), ss.append(s)
    return (torch.cat(q, 1).numpy().astype(np.int64), torch.cat(zs, 1).numpy().astype(np.int64),
            torch.cat(ss, 1))


# ------------------------------------------------------------------ the product
def act64(v, name):
    if name == "silu":
        return v / (1 + np.exp(-v))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return np.maximum(v, 0) if name == "relu" else v


def act_error(v, ev, size, name):
    """Error of the activation at v, its argument off by ev, evaluated in fp32
    (an exponential, a reciprocal and a few products: 16 u of the argument's
    own size, with `size` bounding it)."""
    if name in ("none", "relu"):
        return ev
    return LIP * ev + 16 * U * size


def gemm_ref(x, w, N, alpha=1.0, beta=0.0, y0=None, bias=None, act="none", out="f32"):
    """(value, bound) of the product: x [M, K] a CPU tensor, w a W4Weight."""
    xd, K = f64(x), x.shape[1]
    q, z, s = w4_parts(w, N, K)
    v = alpha * (xd @ ((q - z) * s).T)
    size = abs(alpha) * (np.abs(xd) @ (np.abs(s) * (q + z + 32)).T)
    side = np.zeros_like(v)
    if beta:
        v, side = v + beta * f64(y0), side + np.abs(beta * f64(y0))
    if bias is not None:
        v, side = v + f64(bias), side + np.abs(f64(bias))
    e = gamma(2 * K + 2 * (K // 32 + 1) + 32) * size + 3 * U * side
    val = act64(v, act)
    e = act_error(v, e, size + side, act)
    return val, e + half_step(np.abs(val) + e, out)


# ------------------------------------------------------------------ the layer
def route_ref(logits, k, renormalize=True, scale=1.0):
    """(ids [T, k], weights fp64) with a loop per token."""
    l = f64(logits)
    T, E = l.shape
    ids, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    big = np.finfo(np.float32).max
    for t in range(T):
        row = np.where(np.isnan(l[t]), -np.inf, np.minimum(l[t], big))
        order = [e for e in sorted(range(E), key=lambda e: (-row[e], e)) if row[e] > -np.inf]
        if not order:
            continue
        p = np.exp(np.array([row[e] for e in order]) - row[order[0]])
        p = p[:k] / (p[:k].sum() if renormalize else p.sum())
        ids[t, :len(p)], w[t, :len(p)] = order[:k], scale * p
    return ids, w


def product_ref(x, w, N, K):
    """(x @ W^T, the size that its error goes by, terms) of 16-bit (a tensor
    [N, K]) or 4-bit weights; x fp64 [M, K]."""
    if torch.is_tensor(w):
        wd = f64(w)
        return x @ wd.T, np.abs(x) @ np.abs(wd).T, K
    q, z, s = w4_parts(w, N, K)
    return (x @ ((q - z) * s).T, np.abs(x) @ (np.abs(s) * (q + z + 32)).T,
            2 * K + 2 * (K // 32 + 1))


def moe_ref(x, ids, weights, gate_up, down, I, act, out):
    """(y, bound) fp64 of the layer.  gate_up(e, 0 or 1) and down(e) give an
    expert's matrices.

    Per pair: g and u each within gamma of their sizes; the activation's
    error; h = act(g) u with two roundings, held in two 16-bit numbers (half
    a step twice); the second product, weighted (weights within 16 u), and
    the sum over the choices."""
    xd = f64(x)
    dtype = {torch.float16: "f16", torch.bfloat16: "bf16"}[x.dtype]
    T, H = xd.shape
    y, err = np.zeros((T, H)), np.zeros((T, H))
    rel, least = HALF[dtype]
    for e in np.unique(ids[ids >= 0]):
        t, j = np.nonzero(ids == e)
        g, sg, n1 = product_ref(xd[t], gate_up(e, 0), I, H)
        u, su, _ = product_ref(xd[t], gate_up(e, 1), I, H)
        eg, eu = gamma(n1 + 32) * sg, gamma(n1 + 32) * su
        a = act64(g, act)
        ea = act_error(g, eg, sg, act)
        h = a * u
        eh = np.abs(u) * ea + (np.abs(a) + ea) * eu + 2 * U * np.abs(h)
        eh = eh + np.maximum(rel * rel * (np.abs(h) + eh), least)
        d, sd, n2 = product_ref(h, down(e), H, I)
        _, ed, _ = product_ref(eh, down(e), H, I)       # sizes: eh >= 0
        ed = ed + gamma(n2 + I + 32) * sd * (1 + rel)
        p = np.abs(weights[t, j])[:, None]
        np.add.at(y, t, weights[t, j][:, None] * d)
        np.add.at(err, t, p * (ed + 32 * U * sd))
    return y, err + half_step(np.abs(y) + err, out)


def check(got, value, bound, label=""):
    g = f64(got)
    assert g.shape == value.shape, (g.shape, value.shape)
    bad = ~(np.abs(g - value) <= bound)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(g - value) / bound, -1)), bad.shape)
        raise AssertionError("%s: %d of %d outside the bound; at %s got %r, exact %r, bound %.3g" % (
            label, bad.sum(), bad.size, at, g[at], value[at], bound[at]))
