"""Weights held in 4 bits on the GPU: the format's conversions bit for bit,
the product against the plain 64-bit form within its bound (op_util)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import op_util as ou
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = ou.DT


@pytest.fixture(scope="module")
def tg():
    import dense_gemm_tiled_amd as t
    t.load_library()
    return t


def rand(gen, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(DT[dtype])


# ------------------------------------------------------------------ the format
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_bit_for_bit(tg, src, dtype, group, zeros):
    N, K = 37, 330
    gen = torch.Generator().manual_seed(11)
    w = rand(gen, N, K, dtype=src, scale=0.05)
    w[3] = 0                                              # a row of zeros
    w[4, :] = 0.25                                        # all alike
    w[5, ::2], w[5, 1::2] = 1.0, -1.0                     # both signs equally large
    w[6, :16] = torch.arange(16).to(w.dtype) * 0.5 - 4.0  # ties of the quotient
    w[7] *= 1e-3
    w[8, 40] = float("nan")
    w[9, 70] = float("-inf")
    if src == "f32":
        w[10] = rand(gen, K) * 1e9                        # beyond f16's range
        w[11] = rand(gen, K) * 1e-38                      # scales that vanish or are subnormal
        w[12] = rand(gen, K) * 1e-42
    say("GPU case: quantize", src, dtype, group, zeros)
    got = tg.w4_quantize(w.cuda(), group=group, zeros=zeros, scale_dtype=DT[dtype])
    q, z, s = ou.w4_parts(got, N, K)
    groups = np.arange(K) // group
    rq, rz, rs = ou.quantize_ref(w, group, zeros, dtype)
    assert np.array_equal(s, ou.f64(rs)[:, groups], equal_nan=True)
    assert np.array_equal(z, rz[:, groups])
    assert np.array_equal(q, rq)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 32, True), ("f16", 64, False), ("bf16", 128, False)])
def test_dequantize_rounds_once(tg, out, dtype, group, zeros):
    """Strided output, two matrices; what lies beside the values stays."""
    N, K = 35, 203
    gen = torch.Generator().manual_seed(12)
    w = ou.w4_random(gen, (2,), N, K, dtype, group, zeros, "cuda")
    store = torch.full((2, N + 3, K + 5), 7.0, dtype=DT[out], device="cuda")
    say("GPU case: dequantize", out, dtype, group)
    tg.w4_dequantize(w, store[:, :N, :K])
    for b in range(2):
        v = torch.from_numpy(ou.w4_values([t if t is None else t[b] for t in w], N, K))
        assert torch.equal(store[b, :N, :K].cpu(), v.float().to(DT[out]))
    assert (store[:, N:] == 7).all() and (store[:, :, K:] == 7).all()


@pytest.mark.parametrize("K,group,zeros", [(200, 32, True), (77, 64, False), (256, 128, True)])
def test_pack_lays_out_row_major_codes(tg, K, group, zeros):
    N = 19
    gen = torch.Generator().manual_seed(13)
    q = torch.randint(0, 16, (2, N, K), generator=gen, dtype=torch.uint8)
    padded = torch.nn.functional.pad(q, (0, K % 2))
    rows = padded[..., ::2] | (padded[..., 1::2] << 4)
    G = -(-K // group)
    s = rand(gen, 2, N, G, dtype="f16")
    z = torch.randint(0, 16, (2, N, G), generator=gen, dtype=torch.uint8) if zeros else None
    say("GPU case: pack", K, group, zeros)
    w = tg.w4_pack(rows.cuda(), s.cuda(), None if z is None else z.cuda(), K=K, group=group)
    for b in range(2):
        gq, gz, gs = ou.w4_parts([t if t is None else t[b] for t in w], N, K)
        g = np.arange(K) // group
        assert np.array_equal(gq, q[b].numpy()) and np.array_equal(gs, ou.f64(s[b])[:, g])
        assert np.array_equal(gz, (z[b].numpy()[:, g] if zeros else np.full((N, K), 8)))


def test_quantize_strided_batch_and_rows(tg):
    """Matrices and rows that are not next to each other, at odd addresses."""
    gen = torch.Generator().manual_seed(14)
    store = rand(gen, 3, 40, 300, dtype="bf16").cuda()
    w = store[:, 2:35, 1:258]
    got = tg.w4_quantize(w, group=64)
    ref = tg.w4_quantize(w.contiguous(), group=64)
    assert torch.equal(got.codes, ref.codes) and torch.equal(got.scales, ref.scales)
    with pytest.raises(tg.TcGemmError):
        tg.w4_quantize(store.permute(0, 2, 1), group=64)


# ------------------------------------------------------------------ the product
def run_product(tg, M, N, K, dtype, group, zeros, out=None, seed=1, alpha=1.0, beta=0.0, bias=False,
                act=None, ldx=0, ldy=0, shift=0):
    out = out or dtype
    gen = torch.Generator().manual_seed(seed)
    w = ou.w4_random(gen, (), N, K, dtype, group, zeros, "cuda")
    xs = torch.full((M, (ldx or K) + shift), float("nan"), dtype=DT[dtype])
    xs[:, shift:shift + K] = rand(gen, M, K, dtype=dtype)
    y0 = rand(gen, M, N, dtype=out)
    b = rand(gen, N, dtype=out) if bias else None
    ys = torch.full((M, ldy or N), 7.0, dtype=DT[out], device="cuda")
    y = ys[:, :N]
    if beta:
        y.copy_(y0)
    x = xs.cuda()[:, shift:shift + K]
    say("GPU case: w4_gemm", M, N, K, dtype, group, zeros, out, alpha, beta, bias, act, ldx, ldy, shift)
    r = tg.w4_gemm(x, w, y, alpha=alpha, beta=beta, bias=None if b is None else b.cuda(), activation=act)
    assert r is y
    v, e = ou.gemm_ref(xs[:, shift:shift + K], w, N, alpha, beta, y0, b, act or "none", out)
    ou.check(y, v, e, "w4_gemm")
    assert (ys[:, N:] == 7).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [1, 3, 16, 17, 32, 40, 64, 65, 130])
def test_product(tg, dtype, group, zeros, M):
    run_product(tg, M, 112, 640, dtype, group, zeros, seed=M)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 8), (2, 17, 31), (5, 15, 127), (4, 300, 129),
                                   (20, 33, 130), (33, 31, 255), (70, 129, 385), (200, 70, 1000),
                                   (1, 5000, 96), (3, 9000, 64), (2, 33000, 48), (130, 300, 264)])
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 32, True), ("f16", 128, False)])
def test_product_ragged(tg, M, N, K, dtype, group, zeros):
    run_product(tg, M, N, K, dtype, group, zeros, out="f32", seed=N)


@pytest.mark.parametrize("M", [1, 7, 24, 50, 100])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("act", [None, "relu", "gelu_tanh"])
def test_product_epilogue(tg, M, out, act):
    run_product(tg, M, 75, 300, "bf16", 64, True, out=out, alpha=-0.5, beta=2.0, bias=True, act=act)


@pytest.mark.parametrize("M", [2, 30, 64, 129])
@pytest.mark.parametrize("ldx,ldy,shift", [(301, 80, 0), (304, 75, 1), (311, 99, 3), (8192, 4096, 8)])
def test_product_strides_and_odd_addresses(tg, M, ldx, ldy, shift):
    """Rows of x at any even address; what x holds beside its K columns (NaN
    here) is never read into a result."""
    run_product(tg, M, 75, 300, "f16", 32, False, ldx=ldx, ldy=ldy, shift=shift)


@pytest.mark.parametrize("M,N,K", [(2090, 1010, 264), (33000, 33, 130), (1100, 2000, 1001), (2048, 1024, 128),
                                   (4200, 520, 77), (4200, 1010, 264), (16700, 500, 129), (2048, 4096, 520)])
@pytest.mark.parametrize("dtype,group,zeros,out", [("bf16", 128, False, "bf16"), ("f16", 32, True, "f32"),
                                                   ("bf16", 64, True, "f32"), ("f16", 64, False, "f16"),
                                                   ("bf16", 32, False, "f32"), ("f16", 128, True, "f32")])
def test_product_many_rows(tg, M, N, K, dtype, group, zeros, out):
    """The tiles of long prompts, ragged in every direction."""
    run_product(tg, M, N, K, dtype, group, zeros, out=out, seed=K, bias=True)


def test_product_long_k(tg):
    run_product(tg, 2, 40, 65536, "bf16", 128, False, out="f32")
    run_product(tg, 80, 40, 16400, "f16", 64, True, out="f32")


def test_alpha_zero_reads_neither_operand(tg):
    gen = torch.Generator().manual_seed(5)
    w = ou.w4_random(gen, (), 33, 200, "bf16", 128, False, "cuda")
    for M in (2, 70):
        x = torch.full((M, 200), float("nan"), dtype=torch.bfloat16, device="cuda")
        y = torch.ones(M, 33, dtype=torch.float32, device="cuda")
        tg.w4_gemm(x, w, y, alpha=0.0, beta=0.5)
        assert (y == 0.5).all()


@pytest.mark.parametrize("M", [4, 40, 90])
def test_not_a_number_stays_in_its_row(tg, M):
    gen = torch.Generator().manual_seed(6)
    w = ou.w4_random(gen, (), 50, 260, "f16", 64, True, "cuda")
    x = rand(gen, M, 260, dtype="f16")
    clean = torch.empty(M, 50, dtype=torch.float16, device="cuda")
    tg.w4_gemm(x.cuda(), w, clean)
    x[1, 17], x[M - 1, 259] = float("inf"), float("nan")
    y = torch.empty_like(clean)
    tg.w4_gemm(x.cuda(), w, y)
    bad = torch.isnan(y).all(1).cpu()
    assert bad.nonzero().flatten().tolist() == [1, M - 1]
    assert torch.equal(y[~bad], clean[~bad])


def test_large_offsets(tg):
    """Codes past 4 GiB: rows at both ends of a matrix of 8.6e9 weights, the
    rest of it zero (scale 0)."""
    N, K = 131072 + 5, 65536
    nb, kb = -(-N // 16), K // 128
    codes = torch.zeros(nb, kb, 1024, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(nb, kb, 16, 1, dtype=torch.bfloat16, device="cuda")
    assert codes.numel() > 2 ** 32
    gen = torch.Generator().manual_seed(7)
    ends = ou.w4_random(gen, (2,), 16, K, "bf16", 128, False, "cuda", pad=False)
    blocks = [0, nb - 1]
    for i, b in enumerate(blocks):
        codes[b], scales[b] = ends[0][i, 0], ends[1][i, 0]
    x = rand(gen, 2, K, dtype="bf16")
    y = torch.full((2, N), 7.0, dtype=torch.float32, device="cuda")
    say("GPU case: w4_gemm past 4 GiB")
    tg.w4_gemm(x.cuda(), (codes, scales), y)
    for i, b in enumerate(blocks):
        n = min(16, N - 16 * b)
        v, e = ou.gemm_ref(x, [ends[0][i], ends[1][i], None], n)
        ou.check(y[:, 16 * b:16 * b + n], v, e, "block %d" % b)
    assert (y[:, 16:16 * (nb - 1)] == 0).all()
    back = torch.empty(5, 128, dtype=torch.float32, device="cuda")
    tail = (codes[nb - 1:, kb - 1:].contiguous(), scales[nb - 1:, kb - 1:].contiguous())
    tg.w4_dequantize(tail, back)
    assert np.array_equal(ou.f64(back), ou.w4_values((*tail, None), 5, 128))


def test_same_result_every_time(tg):
    gen = torch.Generator().manual_seed(8)
    for M, N, K in ((1, 2048, 4096), (16, 512, 2048), (64, 512, 1000), (300, 512, 1024)):
        w = ou.w4_random(gen, (), N, K, "bf16", 128, False, "cuda")
        x = rand(gen, M, K, dtype="bf16").cuda()
        a, b = (torch.empty(M, N, dtype=torch.float32, device="cuda") for _ in range(2))
        tg.w4_gemm(x, w, a)
        tg.w4_gemm(x, w, b)
        assert torch.equal(a, b)


# ------------------------------------------------------------------ streams, graphs, refusals
def test_side_stream_and_stream_argument(tg):
    gen = torch.Generator().manual_seed(9)
    dense = rand(gen, 96, 512, dtype="bf16").cuda()
    x = rand(gen, 5, 512, dtype="bf16").cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y1 = torch.empty(5, 96, dtype=torch.bfloat16, device="cuda")
    y2 = torch.empty_like(y1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        w1 = tg.w4_quantize(dense, group=64)
        tg.w4_gemm(x, w1, y1)
    w2 = tg.w4_quantize(dense, group=64, stream=side)
    tg.w4_gemm(x, w2, y2, stream=side)
    side.synchronize()
    v, e = ou.gemm_ref(x.cpu(), w1, 96, out="bf16")
    ou.check(y1, v, e)
    assert torch.equal(y1, y2) and torch.equal(w1.codes, w2.codes)


@pytest.mark.parametrize("M", [1, 48, 200])
def test_captured_and_replayed(tg, M):
    """Two graphs that share the weight, replayed in turn with eager calls
    between them: every replay equals the eager result on its inputs."""
    gen = torch.Generator().manual_seed(10)
    N, K = 256, 1024
    w = tg.w4_quantize(rand(gen, N, K, dtype="f16").cuda(), group=128)
    xs = [rand(gen, M, K, dtype="f16").cuda() for _ in range(2)]
    ys = [torch.zeros(M, N, dtype=torch.float16, device="cuda") for _ in range(2)]
    tg.w4_gemm(xs[0], w, ys[0])
    graphs = []
    for x, y in zip(xs, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tg.w4_gemm(x, w, y, activation="relu")
        graphs.append(g)
    eager = torch.empty_like(ys[0])
    for step in range(4):
        for x, y, g in zip(xs, ys, graphs):
            x.copy_(rand(gen, M, K, dtype="f16"))
            y.zero_()
            g.replay()
            tg.w4_gemm(x, w, eager, activation="relu")
            torch.cuda.synchronize()
            assert torch.equal(y, eager), step


def test_refusals_launch_nothing(tg):
    gen = torch.Generator().manual_seed(15)
    w = tg.w4_quantize(rand(gen, 64, 256, dtype="bf16").cuda())
    x = rand(gen, 4, 256, dtype="bf16").cuda()
    y = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    n0 = tg.dispatch_count()
    bad = [lambda: tg.w4_gemm(x[:, :255], w, y[:, :48]),                  # other blocks
           lambda: tg.w4_gemm(x.half(), w, y), lambda: tg.w4_gemm(x, w, y.half()),
           lambda: tg.w4_gemm(x, w, y[:3]), lambda: tg.w4_gemm(x.cpu(), w, y),
           lambda: tg.w4_gemm(x.t().contiguous().t(), w, y),
           lambda: tg.w4_gemm(x, (w.codes[:, :, :512], w.scales), y),
           lambda: tg.w4_gemm(x, (w.codes, w.scales.float()), y),
           lambda: tg.w4_gemm(x, (w.codes, w.scales, w.codes), y),
           lambda: tg.w4_gemm(x, (w.codes,), y), lambda: tg.w4_gemm(x, w.codes, y),
           lambda: tg.w4_gemm(x, w, y, activation="silu"), lambda: tg.w4_gemm(x, w, y, alpha=math.nan),
           lambda: tg.w4_gemm(x, w, y, bias=torch.zeros(63, dtype=torch.bfloat16, device="cuda")),
           lambda: tg.w4_gemm(x[:0], w, y[:0]),
           lambda: tg.w4_quantize(x, group=16), lambda: tg.w4_quantize(x.to(torch.int8)),
           lambda: tg.w4_quantize(x, scale_dtype=torch.float32), lambda: tg.w4_quantize(x[:0]),
           lambda: tg.w4_quantize(x[0]), lambda: tg.w4_dequantize(w, y),
           lambda: tg.w4_dequantize(w, torch.empty(64, 256, dtype=torch.int32, device="cuda")),
           lambda: tg.w4_pack(w.codes, w.scales)]
    for i, f in enumerate(bad):
        with pytest.raises(tg.TcGemmError):
            f()
            pytest.fail("refusal %d" % i)
    # a view whose allocation ends before the matrix does
    d = tg.QWeightDescT(1, 64, 1 << 20, 128, tg.BF16, False)
    g = tg.QGemmDescT(4, tg.BF16, tg.BF16, 1.0, 0.0, 0, 0)
    ctx, s = tg._torch_stream(0)
    q = tg._w4_ptrs(w)
    st = tg.load_library().tc_qgemm_async(ctx, ctypes.byref(g), ctypes.byref(d), x.data_ptr(), ctypes.byref(q),
                                          y.data_ptr(), None, s)
    assert st in (1, 4)
    assert tg.dispatch_count() == n0
    torch.cuda.synchronize()
    assert (y == 7).all()
