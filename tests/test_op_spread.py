"""The gates of op_spread on the CPU: they pass sums in fp32 and reject what a
broken kernel of the same size would give, at the tests' own sizes."""
import pytest
import torch

import op_spread as sp
import op_util as ou

MATRICES = [("bf16", 128, False), ("f16", 64, True), ("bf16", 32, True)]


def grouped_fp32(x, w, N, K):
    """The kernels' order in fp32: group by group, offset and codes apart."""
    q, z, s = (t.float() for t in sp.parts(w, N, K))
    G, acc = 128 // w[1].shape[-1], torch.zeros(x.shape[0], N)
    for k in range(0, K, G):
        at = slice(k, min(K, k + G))
        c = x[:, at].float() @ (16 + q[:, at]).t() - x[:, at].float() @ (16 + z[:, at]).t()
        acc = acc + s[:, k] * c
    return acc


def test_parts_are_those_of_the_other_reference():
    w = ou.w4_random(torch.Generator().manual_seed(1), (), 21, 150, "f16", 32, True, "cpu")
    for a, b in zip(sp.parts(w, 21, 150), ou.w4_parts(w, 21, 150)):
        assert (a.numpy() == b).all()


@pytest.mark.parametrize("dtype,group,zeros", MATRICES)
@pytest.mark.parametrize("M,N,K", [(2, 40, 65536), (9, 40, 16400), (2, 40, 4096), (3, 30, 77), (1, 1, 1)])
def test_product_gate(dtype, group, zeros, M, N, K):
    gen = torch.Generator().manual_seed(K)
    w = ou.w4_random(gen, (), N, K, dtype, group, zeros, "cpu")
    x = torch.randn(M, K, generator=gen).to(ou.DT[dtype])
    v, var = sp.product(x.double(), w, N, K)
    good = grouped_fp32(x, w, N, K)
    sp.check(good, v, var, "f32")
    sp.check(good.to(ou.DT[dtype]), v, var, dtype)
    q, z, s = sp.parts(w, N, K)
    d = (q - z) * s
    wrong = [torch.zeros_like(v), v * 1.01, v.flip(0) if M > 1 else -v]
    for at in (0, K // 2, K - 1) if K > 128 else ():
        block = slice(at // 128 * 128, at // 128 * 128 + 128)
        lost = v - x[:, block].double() @ d[:, block].t()
        wrong.append(lost)
        one = v.clone()
        one[0, 3] = lost[0, 3] if abs(lost[0, 3] - v[0, 3]) > 0.01 * v.std() else 0
        wrong.append(one)                                  # in a single place
    for bad in wrong:
        with pytest.raises(AssertionError):
            sp.check(bad.float(), v, var, "f32")
    # (a last block that holds a few of 16400 columns is within a half step of bf16: f32 results show it)
    with pytest.raises(AssertionError):
        sp.check(wrong[0].to(ou.DT[dtype]), v, var, dtype)


@pytest.mark.parametrize("dtype,held", [("bf16", (128, False)), ("f16", (64, True)), ("bf16", (32, True)), ("f16", None)])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 9, 130, 5, 3), (1, 2048, 257, 4, 2), (1, 520, 1030, 9, 8), (7, 130, 17, 30, 6),
                                       (33, 96, 130, 2, 2)])
def test_layer_gate(dtype, held, T, H, I, E, k):
    gen = torch.Generator().manual_seed(H + I)
    if held is None:
        up = (torch.randn(E, 2, I, H, generator=gen) * H ** -0.5).to(ou.DT[dtype])
        dn = (torch.randn(E, H, I, generator=gen) * I ** -0.5).to(ou.DT[dtype])
        gu, d = (lambda e, s: up[e, s]), (lambda e: dn[e])
    else:
        up = ou.w4_random(gen, (E, 2), I, H, dtype, *held, "cpu")
        dn = ou.w4_random(gen, (E,), H, I, dtype, *held, "cpu")
        gu = lambda e, s: [t if t is None else t[e, s] for t in up]  # noqa: E731
        d = lambda e: [t if t is None else t[e] for t in dn]  # noqa: E731
    x = torch.randn(T, H, generator=gen).to(ou.DT[dtype])
    ids, w = ou.route_ref(torch.randn(T, E, generator=gen), k)
    ids, w = ids.tolist(), torch.from_numpy(w)

    def fp32(gate_up, ids):
        y = torch.zeros(T, H)
        for t in range(T):
            for j, e in enumerate(ids[t]):
                if e < 0:
                    continue
                m = [(lambda v, n, c, mat: v @ mat.float().t() if torch.is_tensor(mat) else grouped_fp32(v, mat, n, c))(
                    x[t:t + 1].float(), I, H, gate_up(e, s)) for s in (0, 1)]
                h = (torch.nn.functional.silu(m[0]) * m[1])
                o = h @ d(e).float().t() if held is None else grouped_fp32(h, d(e), H, I)
                y[t] += float(w[t, j]) * o[0]
        return y

    y, var = sp.layer(x, ids, w, gu, d, I, "silu", "f32")
    sp.check(fp32(gu, ids), y, var, "f32")
    bf, bvar = sp.layer(x, ids, w, gu, d, I, "silu", dtype)
    sp.check(fp32(gu, ids).to(ou.DT[dtype]), bf, bvar, dtype)
    dropped = [row[:-1] + [-1] for row in ids]
    for bad in (torch.zeros(T, H), fp32(lambda e, s: gu(e, 1 - s), ids), fp32(gu, dropped)):
        for out in ("f32", dtype):
            with pytest.raises(AssertionError):
                sp.check(bad.to(ou.DT[out]), *((y, var) if out == "f32" else (bf, bvar)), out)
