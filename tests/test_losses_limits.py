"""How large the losses' calls may be, on the host, no GPU: what the loss takes
its gradients take, too, or the refusal says why."""
import ctypes

import pytest

import dense_gemm_tiled_amd as tg
from test_losses_host import BIG, LSE, R, S, TG, W, WS, X, cdesc, cgrads, ctx, gsize, lib, size  # noqa: F401


@pytest.mark.parametrize("dtype", [tg.BF16, tg.F16, tg.F32])
@pytest.mark.parametrize("dxt", [True, False, None])
@pytest.mark.parametrize("dwt", [True, False, None])
@pytest.mark.parametrize("T,V,H", [(131072, 32000, 16384), (140001, 300, 16383), (524288, 50000, 4096), (1 << 22, 900, 4096)])
def test_tokens_whose_rows_pass_2_31_elements(lib, T, V, H, dxt, dwt, dtype):  # noqa: F811
    if dxt is dwt is None:
        return
    d = cdesc(T, V, H, dtype)
    # (True: results of x's type, False: f32, None: not wanted)
    g = cgrads(dxt=dtype if dxt else tg.F32, dwt=dtype if dwt else tg.F32)
    g.dx, g.dw = (None if dxt is None else g.dx), (None if dwt is None else g.dw)
    es = 4 if dtype == tg.F32 else 2
    assert size(lib, d)[0] == 0
    st, n = gsize(lib, d, g)
    # a copy of x, and dx's sums where they are not dx itself
    assert st == 0 and n >= T * H * (es + (4 if dxt and es == 2 else 0))


@pytest.mark.parametrize("dtype,T,lddx", [(tg.F32, 1100, 2097120), (tg.BF16, 5000, 500000), (tg.F16, 2000000, 1100)])
def test_rows_of_dx_far_apart(lib, dtype, T, lddx):  # noqa: F811
    assert T * lddx > 2 ** 31
    d, g = cdesc(T, 700, 64, dtype), cgrads(dxt=tg.F32, dwt=dtype, lddx=lddx)
    st, n = gsize(lib, d, g)
    # (words of 16-bit dw are summed in fp32 over the parts of the tokens)
    assert st == 0 and n >= T * 64 * (4 if dtype == tg.F32 else 2) + (0 if dtype == tg.F32 else 700 * 64 * 4)


def test_most_tokens(lib, ctx):  # noqa: F811
    """256 words of G at least: 2^23 - 1 tokens, whatever V is."""
    for V in (1, 64, 255, 256, 257, 1000):
        assert gsize(lib, cdesc((1 << 23) - 1, V, 8), cgrads())[0] == 0, V
        assert gsize(lib, cdesc(1 << 23, V, 8), cgrads())[0] == 3, V
        assert gsize(lib, cdesc(4100000, 515 + V % 16, 8), cgrads())[0] == 0, V
    d, g = cdesc(1 << 23, 64, 8), cgrads()
    assert lib.tc_cross_entropy_backward_async(ctx, R(d), R(g), X, W, TG, LSE, WS, BIG, S) == 3
    assert b"T=8388608" in lib.tc_last_error(ctx)


@pytest.mark.parametrize("dtype", [tg.BF16, tg.F16])
def test_rows_longer_than_their_fp32_sums_may_be(lib, ctx, dtype):  # noqa: F811
    """16-bit rows of up to 8 MiB, whose sums in fp32 take twice that."""
    most = 2097120
    good = [(most, dict(dxt=dtype, dwt=dtype)), (most, dict(dxt=tg.F32, dwt=tg.F32)), (2 * most, dict(dx=None, dwt=dtype))]
    bad = [(most + 8, dict(dxt=dtype, dwt=dtype)), (most + 8, dict(dxt=tg.F32, dw=None)), (most + 8, dict(dx=None, dwt=tg.F32))]
    for H, kw in good:
        assert gsize(lib, cdesc(8, 500, H, dtype), cgrads(**kw))[0] == 0, (H, kw)
    for H, kw in bad:
        d, g = cdesc(8, 500, H, dtype), cgrads(**kw)
        assert gsize(lib, d, g)[0] == 3, (H, kw)
        assert lib.tc_cross_entropy_backward_async(ctx, R(d), R(g), X, W, TG, LSE, WS, BIG, S) == 3
        text = lib.tc_last_error(ctx)
        assert b"%d" % H in text and (b"dx" in text or b"dw" in text), text
    # tokens in parts: a 16-bit dw is summed in fp32, too
    assert gsize(lib, cdesc(1025, 500, most, dtype), cgrads(dx=None, dwt=dtype))[0] == 0
    d, g = cdesc(1025, 500, most + 8, dtype), cgrads(dx=None, dwt=dtype)
    assert gsize(lib, d, g)[0] == 3
    assert lib.tc_cross_entropy_backward_async(ctx, R(d), R(g), X, W, TG, LSE, WS, BIG, S) == 3
    assert b"T=1025" in lib.tc_last_error(ctx)
