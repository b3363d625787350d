"""Long sums of the 4-bit products and expert layers on the GPU, against 64-bit
forms within the spread of fp32 rounding (op_spread): tight where the worst
case of every rounding says little."""
import math

import pytest
import torch

import op_spread as sp
import op_util as ou
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = ou.DT
HELD = [None, (32, True), (64, False), (64, True), (128, False), (128, True), (32, False)]


@pytest.fixture(scope="module")
def tg():
    import dense_gemm_tiled_amd as t
    t.load_library()
    return t


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(gen, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(DT[dtype])


def weight(gen, lead, N, K, dtype, group, zeros):
    """Random codes, scales of either sign and zero points, made on the GPU.
    What the arrays hold past N and K is as random."""
    nb, kb = -(-N // 16), -(-K // 128)
    codes = torch.randint(0, 256, (*lead, nb, kb, 1024), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.rand(*lead, nb, kb, 16, 128 // group, device="cuda", generator=gen) + 0.5
    s = s * torch.where(torch.rand(s.shape, device="cuda", generator=gen) < 0.5, -1.0, 1.0)
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return codes, (s * (0.3 / math.sqrt(K))).to(DT[dtype]), z


# ------------------------------------------------------------------ products
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 128, False), ("f16", 64, True), ("bf16", 32, True),
                                               ("f16", 128, True), ("bf16", 64, False), ("f16", 32, False)])
@pytest.mark.parametrize("M,N,K,kernel", [(2, 40, 65536, "rows"), (16, 600, 16400, "rows"), (80, 40, 16400, "rows"),
                                          (1, 300, 4096, "rows"), (3, 9000, 4093, "rows"), (130, 300, 4096, "rows"),
                                          (300, 8300, 2049, "tile"), (2048, 1056, 4104, "tile")])
def test_product(tg, dtype, group, zeros, M, N, K, kernel):
    gen = generator(M + K)
    w, x = weight(gen, (), N, K, dtype, group, zeros), randn(gen, M, K, dtype=dtype)
    v, var = sp.product(x.double(), w, N, K)
    for out in ("f32", dtype):
        y = torch.full((M, N), 7.0, dtype=DT[out], device="cuda")
        say("GPU case: w4_gemm spread", M, N, K, dtype, group, zeros, out)
        tg.w4_gemm(x, w, y)
        assert tg.last_kernel() == "w4_%s_%s" % (kernel, dtype)
        sp.check(y, v, var, out, "w4_gemm")


def test_product_past_4_gib(tg):
    """Rows at both ends of a matrix of 8.6e9 weights, the rest of it zero."""
    N, K = 131072 + 5, 65536
    nb, kb = -(-N // 16), K // 128
    codes = torch.zeros(nb, kb, 1024, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(nb, kb, 16, 1, dtype=torch.bfloat16, device="cuda")
    gen = generator(7)
    ends = weight(gen, (2,), 16, K, "bf16", 128, False)
    for i, b in enumerate((0, nb - 1)):
        codes[b], scales[b] = ends[0][i, 0], ends[1][i, 0]
    for M in (2, 40):
        x = randn(gen, M, K, dtype="bf16")
        y = torch.full((M, N), 7.0, device="cuda")
        say("GPU case: w4_gemm past 4 GiB", M)
        tg.w4_gemm(x, (codes, scales), y)
        assert tg.last_kernel() == ("w4_rows_bf16" if M == 2 else "w4_tile_bf16")
        for i, b in enumerate((0, nb - 1)):
            n = min(16, N - 16 * b)
            v, var = sp.product(x.double(), (ends[0][i], ends[1][i], None), n, K)
            sp.check(y[:, 16 * b:16 * b + n], v, var, "f32", "block %d" % b)
        assert (y[:, 16:16 * (nb - 1)] == 0).all()


# ------------------------------------------------------------------ layers
def run_layer(tg, T, H, I, E, k, dtype, held, act="silu", seed=1, kernel=None, outs=None):
    gen = generator(seed)
    if held is None:
        up, dn = randn(gen, E, 2, I, H, dtype=dtype, scale=H ** -0.5), randn(gen, E, H, I, dtype=dtype, scale=I ** -0.5)
        gu, d = (lambda e, s: up[e, s]), (lambda e: dn[e])
    else:
        up, dn = weight(gen, (E, 2), I, H, dtype, *held), weight(gen, (E,), H, I, dtype, *held)
        gu = lambda e, s: [t if t is None else t[e, s] for t in up]  # noqa: E731
        d = lambda e: [t if t is None else t[e] for t in dn]  # noqa: E731
    x, l = randn(gen, T, H, dtype=dtype), randn(gen, T, E)
    ids, w = ou.route_ref(l, k)
    ids, w = ids.tolist(), torch.from_numpy(w).cuda()
    for out in outs or ("f32", dtype):
        y = torch.full((T, H), 7.0, dtype=DT[out], device="cuda")
        say("GPU case: moe spread", T, H, I, E, k, dtype, held, act, out)
        tg.moe(x, l, up, dn, y, top_k=k, activation=act, intermediate=I)
        if kernel:
            assert tg.last_kernel() == kernel
        v, var = sp.layer(x, ids, w, gu, d, I, act, out)
        sp.check(y, v, var, out, "moe")


ONE, GENERAL = "moe_one_up+moe_one_down", "moe_sort+moe_up+moe_down+moe_combine"


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,I,E,k", [(9, 130, 5, 3), (24, 385, 4, 2), (100, 128, 3, 3), (2048, 257, 4, 2),
                                     (2049, 200, 4, 2), (2500, 640, 9, 8)])
def test_one_token(tg, H, I, E, k, held, dtype):
    run_layer(tg, 1, H, I, E, k, dtype, held, seed=H + I, kernel=ONE)


@pytest.mark.parametrize("T,H,I,E,k", [(2, 17, 31, 5, 2), (4, 129, 127, 3, 1), (7, 130, 17, 70, 16), (33, 96, 130, 2, 2),
                                       (128, 40, 40, 3, 2), (129, 72, 24, 300, 8), (300, 48, 33, 5, 5),
                                       (3, 600, 257, 16, 8), (16, 300, 300, 512, 4), (24, 2000, 700, 8, 2)])
@pytest.mark.parametrize("dtype,held", [("bf16", None), ("f16", (32, True)), ("bf16", (128, False)), ("f16", (64, True)),
                                        ("bf16", (64, False)), ("f16", None)])
def test_layer(tg, T, H, I, E, k, dtype, held):
    run_layer(tg, T, H, I, E, k, dtype, held, act="gelu_tanh" if T % 2 else "silu", seed=T + H)


@pytest.mark.parametrize("H,I,E,k,dtype,out,kernel", [
    # h of two parts in LDS, in steps of 256 columns (H up to 2048) or 128: 65 and 113 KiB, exactly the 128 KiB it may
    # take with the sums, and past it
    (24, 2048, 9, 8, "f16", "f16", ONE), (24, 14336, 2, 2, "bf16", "bf16", ONE), (24, 32512, 1, 1, "f16", "f16", ONE),
    (24, 32513, 1, 1, "f16", "f16", GENERAL), (24, 4096, 8, 8, "bf16", "bf16", GENERAL),
    (2064, 14336, 2, 2, "f16", "f16", ONE), (2064, 16256, 2, 2, "bf16", "bf16", ONE),
    (2064, 16257, 2, 2, "bf16", "bf16", GENERAL),
    # three parts
    (24, 10752, 2, 2, "bf16", "f32", ONE), (24, 10753, 2, 2, "bf16", "f32", GENERAL), (2064, 2688, 9, 8, "bf16", "f32", ONE),
    (2064, 2689, 9, 8, "bf16", "f32", GENERAL)])
@pytest.mark.parametrize("held", [None, (128, False), (32, True)])
def test_one_token_fills_lds(tg, H, I, E, k, dtype, out, kernel, held):
    run_layer(tg, 1, H, I, E, k, dtype, held, seed=I, kernel=kernel, outs=(out,))


# ------------------------------------------------------------------ ends of the number types
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 128, False), ("f16", 64, True), ("bf16", 32, True)])
@pytest.mark.parametrize("M", [1, 20, 64])
def test_products_of_tiny_and_huge_numbers(tg, dtype, group, zeros, M):
    """Powers of two as factors of x change nothing but the results' exponents:
    x down to its type's subnormal numbers, and up to 2^115 (a group's sums, 128
    times 31 |x| at most, stay inside fp32 up to there)."""
    gen = generator(M)
    N, K = 48, 500
    w = weight(gen, (), N, K, dtype, group, zeros)
    x = torch.randint(-8, 9, (M, K), device="cuda", generator=gen).float()
    ys = []
    for e in (0, -24, 11) if dtype == "f16" else (0, -133, -60, 112):
        y = torch.empty(M, N, device="cuda")
        say("GPU case: w4_gemm scaled", M, dtype, e)
        tg.w4_gemm((x * 2.0 ** e).to(DT[dtype]), w, y)
        ys.append((y.double() * 2.0 ** -e, e))
    for y, e in ys[1:]:
        # (results below 2^-126 are rounded to fp32's subnormal numbers)
        assert torch.allclose(y, ys[0][0], rtol=0, atol=2.0 ** (-150 - e + 10) if e < -100 else 0), e


@pytest.mark.parametrize("group,zeros", [(128, False), (32, True)])
@pytest.mark.parametrize("M", [1, 64])
def test_subnormal_scales(tg, group, zeros, M):
    gen = generator(9)
    N, K = 48, 384
    codes, s, z = weight(gen, (), N, K, "f16", group, zeros)
    s = torch.randint(-1000, 1001, s.shape, device="cuda", generator=gen).float()
    x, ys = randn(gen, M, K, dtype="f16"), []
    for e in (-24, -10):
        y = torch.empty(M, N, device="cuda")
        tg.w4_gemm(x, (codes, (s * 2.0 ** e).half(), z), y)
        ys.append(y * 2.0 ** -e)
    assert torch.equal(*ys) and (ys[0] != 0).any()


@pytest.mark.parametrize("dtype,e", [("f16", -24), ("bf16", -133)])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_layer_reads_subnormal_weights(tg, dtype, e, T):
    """down of subnormal numbers only.  To a matrix instruction they have the
    exponent of the smallest normal number, 2^-14 or 2^-126, so its products
    are added in steps of u of up to |h| times that, whatever the numbers'
    own size: I + 32 sums, each within u |h| 2^-14, against the same numbers
    times 2^24, which are exact to u of their own."""
    gen = generator(T)
    H, I, E, k = 40, 24, 4, 2
    x, l = randn(gen, T, H, dtype=dtype), randn(gen, T, E)
    up = randn(gen, E, 2, I, H, dtype=dtype)
    dn = torch.randint(-8, 9, (E, H, I), device="cuda", generator=gen).float()
    ys = []
    for f in (e, 0):
        y = torch.empty(T, H, device="cuda")
        tg.moe(x, l, up, (dn * 2.0 ** f).to(DT[dtype]), y, top_k=k)
        ys.append(y.double() * 2.0 ** -f)
    ids, p = ou.route_ref(l, k)
    normal = {"f16": 2.0 ** -14, "bf16": 2.0 ** -126}[dtype] * 2.0 ** -e
    for t in range(T):
        bound = 0.0
        for j in range(k):
            g, u = (x[t].double() @ up[ids[t, j], s].double().t() for s in (0, 1))
            h = (sp.activation(g, "silu") * u).abs()
            bound += p[t, j] * (I + 32) * ou.U * float(h.sum()) * (normal + 8)
        assert float((ys[0][t] - ys[1][t]).abs().max()) <= bound
        assert bound < 0.2 * float(ys[1][t].norm()) and float(ys[1][t].norm()) > 0


# ------------------------------------------------------------------ rows past 4 GiB
def test_product_rows_past_4_gib(tg):
    M, N, K = 300000, 24, 8192
    gen = generator(3)
    w = weight(gen, (), N, K, "bf16", 128, False)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    assert x.numel() * 2 > 2 ** 32
    y = torch.full((M, N), 7.0, device="cuda")
    say("GPU case: w4_gemm rows past 4 GiB")
    tg.w4_gemm(x, w, y)
    for at in (slice(0, 130), slice(262140, 262150), slice(M - 70, M)):
        v, var = sp.product(x[at].double(), w, N, K)
        sp.check(y[at], v, var, "f32", str(at))


def test_layer_rows_past_4_gib(tg):
    T, H, I, E, k = 270000, 8192, 16, 2, 1
    gen = generator(4)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    l = randn(gen, T, E)
    up, dn = weight(gen, (E, 2), I, H, "bf16", 128, False), weight(gen, (E,), H, I, "bf16", 128, False)
    y = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    say("GPU case: moe rows past 4 GiB")
    tg.moe(x, l, up, dn, y, top_k=k, intermediate=I)
    for at in (slice(0, 20), slice(262140, 262150), slice(T - 40, T)):
        ids, p = ou.route_ref(l[at], k)
        v, var = sp.layer(x[at], ids.tolist(), torch.from_numpy(p).cuda(),
                          lambda e, s: [t if t is None else t[e, s] for t in up],
                          lambda e: [t if t is None else t[e] for t in dn], I, "silu", "bf16")
        sp.check(y[at], v, var, "bf16", str(at))
