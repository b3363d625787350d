"""4-bit products and expert layers at the ends of their ranges, on the GPU:
which kernels run there, and their results."""
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


@pytest.mark.parametrize("M", [1, 5, 16, 17, 32])
@pytest.mark.parametrize("N", [65536, 65540, 151936])
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 128, False), ("f16", 32, True)])
def test_few_rows_by_a_wide_output(tg, M, N, dtype, group, zeros):
    """A vocabulary's projection while decoding: up to 32 rows never take the
    tiles of 128, however many rows the weight has."""
    gen = torch.Generator().manual_seed(M)
    K = 136
    w = ou.w4_random(gen, (), N, K, dtype, group, zeros, "cuda")
    x = rand(gen, M, K, dtype=dtype)
    y = torch.full((M, N), 7.0, dtype=torch.float32, device="cuda")
    say("GPU case: w4_gemm few rows", M, N, K, dtype, group)
    tg.w4_gemm(x.cuda(), w, y)
    assert tg.last_kernel() == "w4_rows_" + dtype
    v, e = ou.gemm_ref(x, w, N)
    ou.check(y, v, e)


def test_many_rows_take_the_tiles(tg):
    gen = torch.Generator().manual_seed(2)
    w = ou.w4_random(gen, (), 65540, 136, "bf16", 128, False, "cuda")
    x = rand(gen, 33, 136, dtype="bf16")
    y = torch.empty(33, 65540, dtype=torch.bfloat16, device="cuda")
    tg.w4_gemm(x.cuda(), w, y)
    assert tg.last_kernel() == "w4_tile_bf16"
    v, e = ou.gemm_ref(x, w, 65540, out="bf16")
    ou.check(y, v, e)


# ------------------------------------------------------------------ past N and K
def packed(tg, gen, lead, N, K, dtype, group, zeros):
    """Random row-major codes (none of them 8), scales and zero points through w4_pack."""
    q = torch.randint(0, 8, (*lead, N, K + K % 2), generator=gen, dtype=torch.uint8)
    s = rand(gen, *lead, N, -(-K // group), dtype=dtype, scale=K ** -0.5 / 4)
    z = torch.randint(0, 8, s.shape, generator=gen, dtype=torch.uint8) if zeros else None
    return tg.w4_pack((q[..., ::2] | (q[..., 1::2] << 4)).cuda(), s.cuda(), None if z is None else z.cuda(), K=K,
                      group=group)


@pytest.mark.parametrize("N,K", [(1, 1), (33, 40), (40, 203), (16, 256), (19, 129)])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("how", ["quantize", "pack"])
def test_past_the_matrix_stands_for_zero(tg, N, K, group, zeros, how):
    """The whole blocks read as a matrix of their own: zeros past N and K."""
    gen = torch.Generator().manual_seed(N + K)
    say("GPU case: past N and K", N, K, group, zeros, how)
    if how == "pack":
        w = packed(tg, gen, (2,), N, K, "f16", group, zeros)
    else:
        w = tg.w4_quantize(rand(gen, 2, N, K, dtype="f16").cuda() + 1, group=group, zeros=zeros)
    whole = torch.empty(2, -(-N // 16) * 16, -(-K // 128) * 128, device="cuda")
    tg.w4_dequantize(w, whole)
    inside = torch.empty(2, N, K, device="cuda")
    tg.w4_dequantize(w, inside)
    assert torch.equal(whole[:, :N, :K], inside) and (inside != 0).any()
    whole[:, :N, :K] = 0
    assert (whole == 0).all()


@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("H,I", [(64, 33), (72, 40), (130, 121)])
@pytest.mark.parametrize("form", ["library", "tuples", "sized"])
def test_experts_know_their_intermediate_size(tg, T, H, I, form):
    """Experts whose I is no multiple of 16, without `intermediate`: gate_up
    from the quantizer, down from w4_pack (its zero points are not 8); the
    same as plain tuples; and arrays laid out by someone else, whose
    padding holds code 15 and scale NaN, with their sizes."""
    gen = torch.Generator().manual_seed(I)
    E, k, dtype = 5, 2, "f16"
    if form == "sized":
        up = tg.W4Weight(*ou.w4_random(gen, (E, 2), I, H, dtype, 32, True, "cuda"), N=I, K=H)
        dn = tg.W4Weight(*ou.w4_random(gen, (E,), H, I, dtype, 32, True, "cuda"), N=H, K=I)
    else:
        up = tg.w4_quantize(rand(gen, E, 2, I, H, dtype=dtype).cuda() * H ** -0.5 + 0.1, group=32, zeros=True)
        dn = packed(tg, gen, (E,), H, I, dtype, 32, True)
        assert (up.N, up.K, dn.N, dn.K) == (I, H, H, I)
        if form == "tuples":
            up, dn = tuple(up), tuple(dn)
    x, l = rand(gen, T, H, dtype=dtype), rand(gen, T, E)
    y = torch.empty(T, H, device="cuda")
    say("GPU case: moe without intermediate", T, H, I, form)
    tg.moe(x.cuda(), l.cuda(), up, dn, y, top_k=k)
    ids, w = ou.route_ref(l, k)
    one = lambda t, *i: [v if v is None else v[i] for v in t]  # noqa: E731
    v, e = ou.moe_ref(x, ids, w, lambda a, b: one(up, a, b), lambda a: one(dn, a), I, "silu", "f32")
    ou.check(y, v, e)
    # (the elementwise bound is the worst case of every rounding; padding that counted would be 24 % of the
    # whole or more, 7 rows of 121, fp32 sums over groups of 32 are at most gamma_64 * 38 * 0.8 * 32 / 18.7, 2e-4)
    assert np.linalg.norm(ou.f64(y) - v) <= 1e-3 * np.linalg.norm(v)


# ------------------------------------------------------------------ refusals
def test_a_span_too_long_is_refused_for_its_length(tg):
    """An operand that runs past its allocation and over the output that lies
    before it in memory: refused as too long wherever the allocator puts
    things, and without a launch."""
    import ctypes
    lib, (ctx, s) = tg.load_library(), tg._torch_stream(0)
    M, K = 1 << 19, 64
    store = torch.zeros(100 << 20, dtype=torch.uint8, device="cuda")
    end, = (m["address"] + m["total_size"] for m in torch.cuda.memory_snapshot()
            if m["address"] <= store.data_ptr() < m["address"] + m["total_size"])
    out, a = end - (100 << 20), end - (50 << 20)         # [M, 64] 16-bit values are 64 MiB
    b = torch.zeros(K, K, dtype=torch.bfloat16, device="cuda")
    w = tg.w4_quantize(b)
    torch.cuda.synchronize()
    n0 = tg.dispatch_count()
    d = tg.BatchedDescT()
    d.base.M, d.base.N, d.base.K = M, K, K
    d.base.a_dtype = d.base.b_dtype = d.base.c_dtype = tg.BF16
    d.base.accum_dtype, d.base.alpha, d.batch = tg.F32, 1.0, 1
    g = tg.QGemmDescT(M, tg.BF16, tg.BF16, 1.0, 0.0, 0, 0)
    wd, q = tg._w4_desc(w, K, K), tg._w4_ptrs(w)
    R = ctypes.byref
    for x, y, status in ((a, out, 1), (out, a, 1), (out, out + 4096, 4)):
        for call in (lambda: lib.tc_gemm_batched_async(ctx, R(d), x, b.data_ptr(), y, s),
                     lambda: lib.tc_qgemm_async(ctx, R(g), R(wd), x, R(q), y, None, s)):
            assert call() == status, (x, y)
            assert (b"allocation" if status == 1 else b"overlaps") in lib.tc_last_error(ctx)
    assert tg.dispatch_count() == n0
