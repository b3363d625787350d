"""The losses' entry points on the host, no GPU: sizes of workspaces, and every
refusal with its status, before anything is enqueued."""
import ctypes

import pytest

import dense_gemm_tiled_amd as tg

VP = ctypes.c_void_p
P = [0x10000000000 * (i + 1) for i in range(16)]      # distinct, 16-byte aligned, never read
R = ctypes.byref
X, W, TG, LOSS, LSE, WS, S, GRAD, DX, DW, IDS, OUT = P[:12]
BIG = 2 ** 40


@pytest.fixture(scope="module")
def lib():
    return tg.load_library()


@pytest.fixture()
def ctx(lib):
    out = VP()
    assert lib.tc_context_create(R(out)) == 0
    yield out.value
    assert lib.tc_dispatch_count(out.value) == 0
    lib.tc_context_destroy(out.value)


def cdesc(T=64, V=1000, H=128, dtype=tg.BF16, ldx=0, ldw=0, t64=True, scale=1.0):
    return tg.CeDescT(T, V, H, dtype, ldx, ldw, t64, scale)


def cgrads(grad=GRAD, stride=1, dx=DX, dxt=tg.BF16, lddx=0, dw=DW, dwt=tg.BF16, lddw=0, beta=0.0):
    return tg.CeGradsT(grad, stride, dx, dxt, lddx, dw, dwt, lddw, beta)


def size(lib, d, x=X, w=W):
    n = ctypes.c_int64(-1)
    st = lib.tc_cross_entropy_workspace(R(d), x, w, R(n))
    return st, n.value


def gsize(lib, d, g, x=X, w=W):
    n = ctypes.c_int64(-1)
    st = lib.tc_cross_entropy_backward_workspace(R(d), R(g), x, w, R(n))
    return st, n.value


@pytest.mark.parametrize("dtype", [tg.BF16, tg.F16])
@pytest.mark.parametrize("T,V,H", [(1, 1000, 77), (200, 65536, 4095), (300, 500, 1)])
def test_room_for_copied_rows(lib, T, V, H, dtype):
    """Rows that are not whole 16-byte pieces: the copy of W (all of it at these
    sizes) fits beside the gradient of its products."""
    st, odd = gsize(lib, cdesc(T, V, H, dtype), cgrads(dxt=dtype, dwt=dtype))
    assert st == 0 and odd >= (V * ((H + 7) // 8 * 8) + T * V) * 2
    st, odd = size(lib, cdesc(max(T, 257), V, H, dtype))
    assert st == 0 and odd >= (V + max(T, 257)) * ((H + 7) // 8 * 8) * 2


def test_workspaces(lib):
    assert size(lib, cdesc(1, 1, 1))[0] == 0
    st, n = size(lib, cdesc(4096, 131072, 4096))
    assert st == 0 and 0 < n < 64 << 20                    # far from the 2 GiB of all products
    st, n = gsize(lib, cdesc(4096, 131072, 4096), cgrads())
    assert st == 0 and n < 1 << 30
    st, n = size(lib, cdesc(4096, 131072, 1024, tg.F32))
    assert st == 0 and n < 320 << 20
    # one of the two gradients needs no more than both
    both = gsize(lib, cdesc(), cgrads())[1]
    assert gsize(lib, cdesc(), cgrads(dx=None))[1] <= both and gsize(lib, cdesc(), cgrads(dw=None))[1] <= both
    assert lib.tc_cross_entropy_workspace(R(cdesc()), X, W, None) == 1
    n = ctypes.c_int64()
    r = tg.RouteDescT(100, 64, 2, tg.F32, 0, True, 1.0)
    assert lib.tc_moe_balance_workspace(R(r), R(n)) == 0 and n.value > 0
    assert lib.tc_moe_balance_workspace(R(r), None) == 1


BAD = [("T", dict(T=0), 1), ("V", dict(V=-1), 1), ("H", dict(H=0), 1), ("int8", dict(dtype=tg.I8), 2),
       ("scale 0", dict(scale=0.0), 1), ("scale", dict(scale=float("nan")), 1), ("ldx", dict(ldx=127), 1),
       ("ldw", dict(ldw=100), 1), ("ldx long", dict(ldx=1 << 22), 3), ("H long", dict(H=1 << 22), 3),
       ("f32 long", dict(H=1 << 21, dtype=tg.F32), 3), ("tiles", dict(T=1 << 23, V=1 << 20), 3),
       ("T long", dict(T=2 ** 31 - 1), 3)]


@pytest.mark.parametrize("name,kw,status", BAD, ids=[b[0] for b in BAD])
def test_bad_descriptor(lib, ctx, name, kw, status):
    d, g = cdesc(**kw), cgrads()
    g.dx_dtype = g.dw_dtype = d.dtype if d.dtype != tg.I8 else tg.BF16
    assert size(lib, d)[0] == status and gsize(lib, d, g)[0] == status
    assert lib.tc_cross_entropy_async(ctx, R(d), X, W, TG, LOSS, LSE, WS, BIG, S) == status
    assert lib.tc_last_error(ctx) != b""
    assert lib.tc_cross_entropy_backward_async(ctx, R(d), R(g), X, W, TG, LSE, WS, BIG, S) == status
    assert lib.tc_last_error(ctx) != b""


def test_bad_loss_arguments(lib, ctx):
    d = cdesc()
    n = size(lib, d)[1]
    call = lambda *a: lib.tc_cross_entropy_async(ctx, *a)  # noqa: E731
    good = [R(d), X, W, TG, LOSS, LSE, WS, n, S]
    for i in (1, 2, 3, 4, 5, 6, 8):
        assert call(*[None if j == i else v for j, v in enumerate(good)]) == 1, i
    assert call(None, *good[1:]) == 1
    assert lib.tc_cross_entropy_async(None, *good) == 1
    for i, v in ((1, X + 1), (2, W + 1), (3, TG + 4), (4, LOSS + 2), (5, LSE + 1), (6, WS + 8), (7, n - 1), (7, -1)):
        assert call(*[v if j == i else w for j, w in enumerate(good)]) == 1, i
    for i, v in ((4, X + 64), (5, LOSS + 128), (6, W), (4, TG), (6, LSE - 16), (5, W + 1000 * 256 - 4)):
        assert call(*[v if j == i else w for j, w in enumerate(good)]) == 4, i


def test_bad_gradient_arguments(lib, ctx):
    d, g = cdesc(), cgrads()
    n = gsize(lib, d, g)[1]
    call = lambda *a: lib.tc_cross_entropy_backward_async(ctx, *a)  # noqa: E731
    good = [R(d), R(g), X, W, TG, LSE, WS, n, S]
    for i in (2, 3, 4, 5, 6, 8):
        assert call(*[None if j == i else v for j, v in enumerate(good)]) == 1, i
    assert call(None, *good[1:]) == 1 and call(R(d), None, *good[2:]) == 1
    assert lib.tc_cross_entropy_backward_async(None, *good) == 1
    for i, v in ((5, LSE + 2), (6, WS + 4), (7, n - 1)):
        assert call(*[v if j == i else w for j, w in enumerate(good)]) == 1, i
    for kw, status in ((dict(dx=None, dw=None), 1), (dict(grad=None), 1), (dict(grad=GRAD + 2), 1),
                       (dict(stride=-1), 1), (dict(stride=2 ** 31), 1), (dict(dxt=tg.F16), 2),
                       (dict(dwt=tg.I8), 2), (dict(lddx=127), 1), (dict(lddw=-5), 1), (dict(dx=DX + 1), 1),
                       (dict(dwt=tg.F32, dw=DW + 2), 1), (dict(beta=float("inf")), 1), (dict(lddw=1 << 22), 3),
                       (dict(dx=X), 4), (dict(dw=W + 256), 4), (dict(dx=DW), 4), (dict(dw=GRAD), 4),
                       (dict(dx=LSE), 4), (dict(dw=WS), 4)):
        b = cgrads(**kw)
        assert call(R(d), R(b), *good[2:7], BIG // 2, S) == status, kw
    # no room for 256 words at a time
    assert gsize(lib, cdesc(T=1 << 23, V=64, H=8), cgrads())[0] in (0, 3)
    assert gsize(lib, cdesc(T=(1 << 24) - 16, V=512, H=8), cgrads())[0] == 3


ROUTE = [("T", dict(T=0), 1), ("E", dict(E=0), 1), ("k", dict(k=0), 1), ("experts", dict(E=513), 2),
         ("choices", dict(k=17), 2), ("more choices than experts", dict(E=4, k=5), 2), ("int8", dict(dtype=tg.I8), 2),
         ("ld", dict(ld=63), 1), ("T long", dict(T=2 ** 31 - 1), 3)]


def rdesc(T=100, E=64, k=2, dtype=tg.BF16, ld=0, scale=1.0):
    return tg.RouteDescT(T, E, k, dtype, ld, True, scale)


@pytest.mark.parametrize("name,kw,status", ROUTE, ids=[b[0] for b in ROUTE])
def test_bad_router(lib, ctx, name, kw, status):
    r, n = rdesc(**kw), ctypes.c_int64()
    assert lib.tc_moe_balance_workspace(R(r), R(n)) == status
    assert lib.tc_moe_balance_async(ctx, R(r), X, IDS, 1.0, LOSS, OUT, LSE, WS, BIG, S) == status
    assert lib.tc_last_error(ctx) != b""
    assert lib.tc_moe_route_backward_async(ctx, R(r), X, IDS, GRAD, None, None, DX, tg.F32, 0, S) == status


def test_bad_router_arguments(lib, ctx):
    r, n = rdesc(), ctypes.c_int64()
    assert lib.tc_moe_balance_workspace(R(r), R(n)) == 0
    good = [R(r), X, IDS, 1.0, LOSS, OUT, LSE, WS, n.value, S]
    call = lambda *a: lib.tc_moe_balance_async(ctx, *a)  # noqa: E731
    for i in (0, 1, 2, 4, 5, 6, 7, 9):
        assert call(*[None if j == i else v for j, v in enumerate(good)]) == 1, i
    for i, v in ((1, X + 1), (2, IDS + 2), (3, float("nan")), (4, LOSS + 1), (5, OUT + 2), (6, LSE + 3), (7, WS + 8),
                 (8, n.value - 1)):
        assert call(*[v if j == i else w for j, w in enumerate(good)]) == 1, i
    for i, v in ((4, X), (5, IDS + 796), (6, OUT + 252), (7, X + 12799 // 16 * 16)):
        assert call(*[v if j == i else w for j, w in enumerate(good)]) == 4, i
    good = [R(r), X, IDS, GRAD, LSE, LOSS, DX, tg.BF16, 0, S]
    call = lambda *a: lib.tc_moe_route_backward_async(ctx, *a)  # noqa: E731
    for i in (0, 1, 2, 4, 5, 6, 9):
        assert call(*[None if j == i else v for j, v in enumerate(good)]) == 1, i
    assert call(R(r), X, IDS, None, None, None, DX, tg.BF16, 0, S) == 1
    assert call(R(rdesc(scale=float("inf"))), *good[1:]) == 1
    for i, v, status in ((3, GRAD + 2, 1), (4, LSE + 1, 1), (5, LOSS + 2, 1), (6, DX + 1, 1), (7, tg.F16, 2),
                         (7, tg.I32, 2), (8, 63, 1), (6, X + 128, 4), (6, IDS, 4), (6, GRAD + 400, 4), (6, LSE, 4),
                         (6, LOSS, 4)):
        assert call(*[v if j == i else w for j, w in enumerate(good)]) == status, (i, v)


@pytest.mark.parametrize("E,most", [(8, 256), (16, 256), (17, 128), (32, 128), (33, 64), (64, 64), (512, 64)])
def test_few_tokens_need_no_workspace(lib, E, most):
    n = ctypes.c_int64(-1)
    assert lib.tc_moe_balance_workspace(R(rdesc(T=most, E=E)), R(n)) == 0 and n.value == 0
    assert lib.tc_moe_balance_workspace(R(rdesc(T=most + 1, E=E)), R(n)) == 0 and n.value > 0
