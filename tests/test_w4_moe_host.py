"""The 4-bit weight and mixture-of-experts entry points on the host, no GPU:
sizes, and every refusal with its status, before anything is enqueued."""
import ctypes

import pytest
import torch

import dense_gemm_tiled_amd as tg

VP = ctypes.c_void_p
P = [0x10000000000 * (i + 1) for i in range(16)]      # distinct, 16-byte aligned, never read


@pytest.fixture(scope="module")
def lib():
    return tg.load_library()


@pytest.fixture()
def ctx(lib):
    out = VP()
    assert lib.tc_context_create(ctypes.byref(out)) == 0
    yield out.value
    assert lib.tc_dispatch_count(out.value) == 0
    lib.tc_context_destroy(out.value)


def wdesc(batch=1, N=64, K=256, group=128, dtype=tg.BF16, zeros=False):
    return tg.QWeightDescT(batch, N, K, group, dtype, zeros)


def weight(zeros=False, codes=P[0], scales=P[1]):
    return tg.QWeightT(codes, scales, P[2] if zeros else None)


@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (16, 128, 128), (17, 129, 64), (4099, 4093, 32)])
@pytest.mark.parametrize("zeros", [False, True])
def test_sizes(lib, N, K, group, zeros):
    c, s, z = (ctypes.c_int64() for _ in range(3))
    d = wdesc(3, N, K, group, zeros=zeros)
    assert lib.tc_qweight_sizes(ctypes.byref(d), ctypes.byref(c), ctypes.byref(s), ctypes.byref(z)) == 0
    blocks = 3 * -(-N // 16) * -(-K // 128)
    assert c.value == blocks * 1024
    assert s.value == blocks * 16 * (128 // group) * 2
    assert z.value == (s.value // 2 if zeros else 0)
    assert lib.tc_qweight_sizes(ctypes.byref(d), None, None, None) == 0


BAD_WEIGHT = [("batch", dict(batch=0), 1), ("N", dict(N=0), 1), ("K", dict(K=-1), 1),
              ("group", dict(group=48), 1), ("group 0", dict(group=0), 1), ("f32", dict(dtype=tg.F32), 2),
              ("K long", dict(K=1 << 22), 3),
              ("blocks", dict(batch=2 ** 31 - 1, N=2 ** 31 - 1, K=128), 3)]


@pytest.mark.parametrize("name,kw,status", BAD_WEIGHT, ids=[b[0] for b in BAD_WEIGHT])
def test_bad_weight_descriptor(lib, ctx, name, kw, status):
    d, w = wdesc(**kw), weight()
    assert lib.tc_qweight_sizes(ctypes.byref(d), None, None, None) == status
    g = tg.QGemmDescT(4, tg.BF16, tg.BF16, 1.0, 0.0, 0, 0)
    assert lib.tc_quantize_async(ctx, ctypes.byref(d), P[4], tg.F32, 0, 0, ctypes.byref(w), P[9]) == status
    assert lib.tc_last_error(ctx) != b""
    assert lib.tc_dequantize_async(ctx, ctypes.byref(d), ctypes.byref(w), P[4], tg.F32, 0, 0, P[9]) == status
    assert lib.tc_qweight_pack_async(ctx, ctypes.byref(d), ctypes.byref(w), ctypes.byref(w), P[9]) == status
    assert lib.tc_qgemm_async(ctx, ctypes.byref(g), ctypes.byref(d), P[4], ctypes.byref(w), P[5], None,
                              P[9]) == status


def test_bad_format_arguments(lib, ctx):
    d, w = wdesc(), weight()
    R, B = ctypes.byref, P[9]
    q = lambda *a: lib.tc_quantize_async(ctx, *a)  # noqa: E731
    assert q(None, P[4], tg.F32, 0, 0, R(w), B) == 1
    assert q(R(d), None, tg.F32, 0, 0, R(w), B) == 1
    assert q(R(d), P[4], tg.F32, 0, 0, None, B) == 1
    assert q(R(d), P[4], tg.F32, 0, 0, R(w), None) == 1
    assert q(R(d), P[4], tg.I8, 0, 0, R(w), B) == 2
    assert q(R(d), P[4], tg.F32, 255, 0, R(w), B) == 1
    assert q(R(d), P[4], tg.F32, 2 ** 62, 0, R(w), B) == 3
    assert q(R(wdesc(batch=2)), P[4], tg.F32, 0, 64 * 256 - 1, R(w), B) == 1
    assert q(R(d), P[4], tg.F32, 0, 0, R(tg.QWeightT(None, P[1], None)), B) == 1
    assert q(R(d), P[4], tg.F32, 0, 0, R(weight(zeros=True)), B) == 1          # zeros not described
    assert q(R(wdesc(zeros=True)), P[4], tg.F32, 0, 0, R(w), B) == 1
    assert q(R(d), P[4], tg.F32, 0, 0, R(weight(codes=P[0] + 8)), B) == 1      # alignment
    assert q(R(d), P[0] + 64, tg.F32, 0, 0, R(w), B) == 4                      # W overlaps codes
    assert q(R(d), P[4], tg.F32, 0, 0, R(weight(scales=P[0] + 1024)), B) == 4
    dq = lambda *a: lib.tc_dequantize_async(ctx, *a)  # noqa: E731
    assert dq(R(d), R(w), P[0] + 4096, tg.F32, 0, 0, B) == 4
    assert dq(R(d), R(w), P[4], tg.I32, 0, 0, B) == 2
    assert dq(R(d), R(w), P[4], tg.F32, 100, 0, B) == 1
    pk = lambda *a: lib.tc_qweight_pack_async(ctx, *a)  # noqa: E731
    assert pk(R(d), None, R(w), B) == 1
    assert pk(R(d), R(weight(scales=P[5] + 1)), R(w), B) == 1
    assert pk(R(d), R(weight(codes=P[0] + 7)), R(w), B) == 4
    assert lib.tc_quantize_async(None, R(d), P[4], tg.F32, 0, 0, R(w), B) == 1


def test_bad_product(lib, ctx):
    R = ctypes.byref
    d, w = wdesc(), weight()

    def call(g=None, d=d, x=P[4], w=w, y=P[5], ep=None, s=P[9]):
        g = g or tg.QGemmDescT(4, tg.BF16, tg.BF16, 1.0, 0.0, 0, 0)
        return lib.tc_qgemm_async(ctx, R(g), R(d), x, R(w), y, R(ep) if ep else None, s)

    Q = tg.QGemmDescT
    assert call(x=None) == call(y=None) == call(s=None) == 1
    assert call(d=wdesc(batch=2)) == 2
    for g, status in [(Q(0, 2, 2, 1, 0, 0, 0), 1), (Q(4, 1, 1, 1, 0, 0, 0), 2), (Q(4, 2, 1, 1, 0, 0, 0), 2),
                      (Q(4, 0, 0, 1, 0, 0, 0), 2), (Q(4, 2, 2, float("nan"), 0, 0, 0), 1),
                      (Q(4, 2, 2, 1, float("inf"), 0, 0), 1), (Q(4, 2, 2, 1, 0, 255, 0), 1),
                      (Q(4, 2, 2, 1, 0, 0, 63), 1), (Q(4, 2, 2, 1, 0, 1 << 22, 0), 3),
                      (Q(65535 * 16 + 1, 2, 2, 1, 0, 0, 0), 3)]:
        assert call(g) == status, (g.M, g.x_dtype, status)
    assert call(x=P[4] + 1) == 1 and call(y=P[5] + 1) == 1
    assert call(Q(4, 2, 0, 1, 0, 0, 0), y=P[5] + 2) == 1
    assert call(y=P[4] + 100) == 4 and call(y=P[0] + 4096) == 4 and call(y=P[1]) == 4
    E = tg.EpilogueT
    assert call(ep=E(None, 0, 7, None, 0)) == 1
    assert call(ep=E(None, 0, 3, None, 0)) == 1
    assert call(ep=E(None, 0, 0, P[6], 0)) == 2
    assert call(ep=E(P[5] + 2, 0, 0, None, 0)) == 4


def rdesc(T=5, E=16, k=2, dtype=tg.F32, ld=0, renorm=True, scale=1.0):
    return tg.RouteDescT(T, E, k, dtype, ld, renorm, scale)


BAD_ROUTE = [("T", dict(T=0), 1), ("E", dict(E=0), 1), ("k", dict(k=0), 1), ("k>E", dict(k=5, E=4), 2),
             ("E>512", dict(E=513), 2), ("k>16", dict(k=17, E=64), 2), ("i8", dict(dtype=tg.I8), 2),
             ("ld", dict(ld=15), 1), ("scale", dict(scale=float("inf")), 1)]


@pytest.mark.parametrize("name,kw,status", BAD_ROUTE, ids=[b[0] for b in BAD_ROUTE])
def test_bad_route(lib, ctx, name, kw, status):
    r = rdesc(**kw)
    assert lib.tc_moe_route_async(ctx, ctypes.byref(r), P[0], P[1], P[2], P[9]) == status


def test_bad_route_pointers(lib, ctx):
    r = rdesc()
    f = lambda *a: lib.tc_moe_route_async(ctx, ctypes.byref(r), *a)  # noqa: E731
    assert f(None, P[1], P[2], P[9]) == f(P[0], None, P[2], P[9]) == f(P[0], P[1], P[2], None) == 1
    assert f(P[0] + 2, P[1], P[2], P[9]) == 1 and f(P[0], P[1] + 2, P[2], P[9]) == 1
    assert f(P[0], P[0] + 4, P[2], P[9]) == 4 and f(P[0], P[1], P[1] + 4, P[9]) == 4
    assert lib.tc_moe_route_async(ctx, None, P[0], P[1], P[2], P[9]) == 1


def mdesc(T=5, H=64, I=48, E=16, k=2, x=tg.BF16, y=tg.BF16, ldx=0, ldy=0, gate=0, group=0, zeros=False):
    return tg.MoeDescT(T, H, I, E, k, x, y, ldx, ldy, gate, group, zeros)


BAD_MOE = [("T", dict(T=0), 1), ("H", dict(H=0), 1), ("I", dict(I=-4), 1), ("E", dict(E=513), 2),
           ("k", dict(k=17, E=100), 2), ("k>E", dict(k=5, E=4), 2), ("x f32", dict(x=tg.F32, y=tg.F32), 2),
           ("y", dict(y=tg.F16), 2), ("gate", dict(gate=2), 1), ("group", dict(group=16), 1),
           ("zeros", dict(zeros=True), 1), ("T long", dict(T=65535 * 128 + 1), 3),
           ("H long", dict(H=1 << 22), 3), ("I long", dict(I=1 << 22), 3)]


# launches whose threads would not fit 32 bits
BAD_MOE += [("T by H", dict(T=1 << 20, H=4352), 3), ("E by I", dict(E=512, I=1 << 20), 3),
            ("E by H", dict(E=512, H=1 << 20), 3)]


@pytest.mark.parametrize("name,kw,status", BAD_MOE, ids=[b[0] for b in BAD_MOE])
def test_bad_layer(lib, ctx, name, kw, status):
    d, n, w = mdesc(**kw), ctypes.c_int64(), tg.QWeightT(P[0], None, None)
    assert lib.tc_moe_workspace(ctypes.byref(d), ctypes.byref(n)) == status
    r = rdesc(T=d.T, E=d.E, k=d.top_k)
    st = lib.tc_moe_async(ctx, ctypes.byref(d), P[3], ctypes.byref(r), P[4], None, None, ctypes.byref(w),
                          ctypes.byref(w), P[5], P[6], 1 << 30, P[9])
    assert st == status
    assert lib.tc_last_error(ctx) != b""


def test_bad_layer_arguments(lib, ctx):
    n = ctypes.c_int64()
    assert lib.tc_moe_workspace(ctypes.byref(mdesc()), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.tc_moe_workspace(ctypes.byref(mdesc()), None) == 1
    dense = lambda p: tg.QWeightT(p, None, None)  # noqa: E731

    def call(d=None, x=P[3], r="fits", logits=P[4], ids=None, weights=None, up=dense(P[0]), down=dense(P[1]),
             y=P[5], ws=P[6], size=n.value, s=P[9]):
        d = d or mdesc()
        r = rdesc(T=d.T, E=d.E, k=d.top_k) if r == "fits" else r
        ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
        return lib.tc_moe_async(ctx, ctypes.byref(d), x, ref(r), logits, ids, weights, ref(up), ref(down), y,
                                ws, size, s)

    assert call(x=None) == call(y=None) == call(s=None) == call(ws=None) == 1
    assert call(up=None) == call(down=None) == call(up=dense(None)) == 1
    assert call(ids=P[7], weights=P[8]) == 1                       # logits too
    assert call(logits=None) == 1 and call(logits=None, r=None, ids=P[7]) == 1
    assert call(r=rdesc(T=4)) == 1 and call(r=rdesc(E=15)) == 1 and call(r=rdesc(k=1)) == 1
    assert call(r=None) == 1 and call(r=rdesc(dtype=tg.I8)) == 2
    assert call(size=n.value - 1) == 1 and call(ws=P[6] + 8) == 1
    assert call(d=mdesc(ldx=63)) == 1 and call(d=mdesc(ldy=63)) == 1 and call(d=mdesc(ldx=1 << 22)) == 3
    assert call(x=P[3] + 1) == 1 and call(logits=P[4] + 2) == 1 and call(up=dense(P[0] + 1)) == 1
    assert call(logits=None, r=None, ids=P[7] + 2, weights=P[8]) == 1
    assert call(up=weight()) == 1                                  # scales with 16-bit weights
    assert call(d=mdesc(group=64), up=weight(), down=dense(P[7])) == 1
    assert call(d=mdesc(group=64, zeros=True), up=weight(), down=weight()) == 1
    assert call(d=mdesc(group=64), up=weight(codes=P[0] + 8), down=weight()) == 1
    assert call(y=P[3] + 100) == 4 and call(y=P[6] + 256) == 4 and call(ws=P[0] + 1024) == 4
    assert call(y=P[0] + 4096) == 4 and call(ws=P[4]) == 4


def test_python_refusals_without_a_gpu():
    import torch
    x, y = torch.zeros(2, 64), torch.zeros(2, 64)
    for f in (lambda: tg.w4_quantize(x), lambda: tg.moe_route(x, 2), lambda: tg.w4_dequantize((x, x), y),
              lambda: tg.w4_gemm(x, (x, x), y), lambda: tg.w4_pack(x, x), lambda: tg.moe(x, y, x, x, y)):
        with pytest.raises(tg.TcGemmError):
            f()


def test_grids_past_32_bits(lib, ctx):
    """Refused before anything is launched; at the limit (2^24 - 16 workgroups
    of 256 threads: 16 (2^20 - 1) for T and H here) the host's
    checks pass (sizes only, no launch)."""
    n = ctypes.c_int64()
    assert lib.tc_moe_workspace(ctypes.byref(mdesc(T=(1 << 20) - 1, H=4080)), ctypes.byref(n)) == 0
    r = rdesc(T=1 << 27)
    assert lib.tc_moe_route_async(ctx, ctypes.byref(r), P[0], P[1], P[2], P[9]) == 3
    d = wdesc(N=1 << 28, K=16)
    assert lib.tc_qweight_sizes(ctypes.byref(d), None, None, None) == 3
    d = wdesc(N=(1 << 28) - 256, K=16)
    assert lib.tc_qweight_sizes(ctypes.byref(d), None, None, None) == 0
    d, w = wdesc(N=1 << 18, K=16), weight()
    g = tg.QGemmDescT(65535 * 16, d.scale_dtype, d.scale_dtype, 1.0, 0.0, 0, 0)
    assert lib.tc_qgemm_async(ctx, ctypes.byref(g), ctypes.byref(d), P[3], ctypes.byref(w), P[4], None, P[9]) == 3


def test_broadcast_operands_refused():
    """A stride of 0 means contiguous to the library: rows or matrices that
    are broadcast would be read past the end of the tensor."""
    row, w = torch.zeros(1, 128), tg.W4Weight(torch.zeros(1, 1, 1024, dtype=torch.uint8),
                                              torch.zeros(1, 1, 16, 1, dtype=torch.bfloat16))
    x, y = row.bfloat16().expand(4, 128), torch.zeros(4, 16, dtype=torch.bfloat16)
    for f in (lambda: tg._make_qgemm(x, tuple(w), y, 1.0, 0.0),
              lambda: tg._make_qgemm(x.contiguous(), tuple(w), y[:1].expand(4, 16), 1.0, 0.0),
              lambda: tg._make_route(row.expand(4, 128), 2, True, 1.0),
              lambda: tg._dense_batch(row.expand(4, 128), "w"),
              lambda: tg._dense_batch(torch.zeros(1, 3, 128).expand(2, 3, 128), "w"),
              lambda: tg._dense_batch(torch.zeros(3, 128).expand(2, 2, 3, 128), "w")):
        with pytest.raises(tg.TcGemmError, match="broadcast"):
            f()
    # one row, or one matrix, has no pitch to get wrong
    tg._make_qgemm(row.bfloat16().expand(1, 128), tuple(w), y[:1], 1.0, 0.0)
    assert tg._dense_batch(torch.zeros(3, 128).expand(1, 3, 128), "w")[3:] == (128, 0)
