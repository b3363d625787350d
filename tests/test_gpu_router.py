"""A router's balance loss and the gradient of its logits against 64 bits
(loss_util has the bounds)."""
import math

import pytest
import torch

import dense_gemm_tiled_amd as tg
import loss_util as lu

pytestmark = pytest.mark.gpu


def case(T, E, k, dtype, seed=1, dead=0.1, gone=0.02, pad=0, spread=1.0):
    """logits with some experts masked and some tokens padded (NaN logits, no
    ids), and the experts of each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = spread * torch.randn(T, E, device="cuda", generator=g)
    logits[torch.rand(T, E, device="cuda", generator=g) < gone] = -math.inf
    logits = logits.to(lu.DT[dtype])
    if pad:
        whole = torch.full((T, E + pad), float("nan"), dtype=logits.dtype, device="cuda")
        whole[:, :E] = logits
        logits = whole[:, :E]
    ids, _ = tg.moe_route(logits, k)
    out = torch.rand(T, device="cuda", generator=g) < dead
    ids[out] = -1
    logits[out] = float("nan")
    return logits, ids, g


def balance(logits, ids, coef=0.25, **kw):
    loss, counts, slope = tg.moe_balance(logits, ids, coef=coef, **kw)
    want, n, sl, off, soff = lu.balance64(logits, ids, coef)
    assert loss.shape == () and counts.dtype == torch.int32 and torch.equal(counts.long(), n)
    assert abs(float(loss.double() - want)) <= off + 2.0 ** -24 * abs(float(want))
    assert ((slope.double() - sl).abs() <= soff + 2.0 ** -24 * sl.abs()).all()
    return loss, counts, slope


def gradient(logits, ids, dweights, renormalize=True, scale=1.0, slope=None, dloss=None, out=None, pad=0, **kw):
    T, E = logits.shape
    kind = out or lu.NAME[logits.dtype]
    whole = torch.full((T, E + pad), float("nan"), dtype=lu.DT[kind], device="cuda")
    d = whole[:, :E]
    got = tg.moe_route_backward(logits, ids, dweights, d, renormalize=renormalize, scale=scale, slope=slope,
                                dloss=dloss, **kw)
    assert got is d
    value, off = lu.route_grad64(logits, ids, dweights, renormalize, scale, slope, dloss)
    lu.check(d, value, off, None, kind, "dlogits")
    assert torch.isnan(whole[:, E:]).all()
    _, p, _, _ = lu.router64(logits, ids)
    assert (d[p == 0] == 0).all()
    return d


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (61, 8, 2), (64, 64, 6), (65, 60, 4), (130, 61, 7), (200, 128, 8),
         (1021, 33, 3), (257, 256, 8), (90, 250, 16), (300, 512, 10), (77, 509, 9), (5000, 12, 2)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_balance(T, E, k, dtype):
    logits, ids, _ = case(T, E, k, dtype, seed=T + E)
    balance(logits, ids)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route_gradient(T, E, k, dtype, renormalize):
    logits, ids, g = case(T, E, k, dtype, seed=T + E + 1)
    dw = torch.randn(T, k, device="cuda", generator=g)
    slope = torch.randn(E, device="cuda", generator=g)
    dloss = torch.full((), 0.7, device="cuda")
    gradient(logits, ids, dw, renormalize, 2.5, slope, dloss)
    gradient(logits, ids, dw, renormalize)
    gradient(logits, ids, None, renormalize, 1.0, slope, dloss, out="f32")


@pytest.mark.parametrize("T,E", [(100000, 64), (40000, 256), (20000, 17)])
def test_many_tokens(T, E):
    logits, ids, g = case(T, E, 4, "bf16")
    balance(logits, ids)
    gradient(logits, ids, torch.randn(T, 4, device="cuda", generator=g), slope=torch.randn(E, device="cuda"),
             dloss=torch.ones((), device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,pad", [(64, 4), (64, 3), (60, 1), (256, 8)])
def test_pitches_and_addresses(E, pad, dtype):
    logits, ids, g = case(150, E, 4, dtype, pad=pad)
    dw = torch.randn(150, 4, device="cuda", generator=g)
    balance(logits, ids)
    gradient(logits, ids, dw, pad=pad)
    gradient(logits, ids, dw, pad=1)
    balance(logits[1:], ids[1:])
    gradient(logits[1:], ids[1:].contiguous(), dw[1:].contiguous())
    odd = torch.empty(150 * E + 1, dtype=logits.dtype, device="cuda")[1:].view(150, E).copy_(logits)
    balance(odd, ids)
    gradient(odd, ids, dw, pad=pad)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_with_little_left(dtype):
    """Tokens with no finite logit, with one, with infinities, with the type's
    lowest value, with ids outside, twice the same and fewer than top_k."""
    E, k = 12, 3
    low = torch.finfo(lu.DT[dtype]).min
    logits = torch.randn(10, E, device="cuda").to(lu.DT[dtype])
    logits[0] = -math.inf
    logits[1] = math.nan
    logits[2] = -math.inf
    logits[2, 5] = 1.0
    logits[3, 4] = math.inf
    logits[4] = low
    logits[5, ::2] = low
    logits[6, 1:4] = math.nan
    ids = torch.tensor([[0, 1, 2], [3, 4, 5], [5, -1, -1], [4, 1, 0], [0, 1, 2], [1, 3, 5], [0, 5, 1],
                        [3, 3, 7], [-1, E, 2 ** 31 - 1], [-5, 2, E + 7]], dtype=torch.int32, device="cuda")
    dw = torch.randn(10, k, device="cuda")
    dw[8] = math.nan
    dw[9, 0] = math.nan
    dw[9, 2] = math.inf
    dw[2, 1:] = math.nan
    dw[6, 2] = math.nan                       # (the place of a logit that is no number)
    slope, dloss = torch.randn(E, device="cuda"), torch.full((), -1.5, device="cuda")
    balance(logits, ids)
    for renormalize in (True, False):
        d = gradient(logits, ids, dw, renormalize, 1.5, slope, dloss)
        assert (d[[0, 1, 8]] == 0).all()
        gradient(logits, ids, dw, renormalize, 1.5, out="f32")


def test_no_token_counts():
    logits = torch.full((70, 16), float("nan"), device="cuda")
    ids = torch.full((70, 2), -1, dtype=torch.int32, device="cuda")
    loss, counts, slope = balance(logits, ids)
    assert float(loss) == 0 and (counts == 0).all() and (slope == 0).all()
    d = tg.moe_route_backward(logits, ids, torch.full((70, 2), float("nan"), device="cuda"), torch.empty_like(logits),
                              slope=slope, dloss=loss)
    assert (d == 0).all()


def test_balanced_and_collapsed():
    """Every expert chosen alike: the loss is coef and the slopes are 0.  All
    tokens on one expert: E times its probability."""
    T, E = 512, 16
    logits = torch.zeros(T, E, device="cuda")
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % E)[:, None].contiguous()
    loss, counts, slope = balance(logits, ids, coef=0.5)
    assert float(loss) == 0.5 and (counts == T // E).all() and (slope == 0).all()
    logits[:, 3] = math.inf
    loss, counts, slope = balance(logits, torch.full((T, 1), 3, dtype=torch.int32, device="cuda"), coef=0.5)
    assert float(loss) == 0.5 * E and int(counts[3]) == T


def test_gradient_against_differences():
    """Central differences of moe_balance's loss and of moe_route's weights
    (their choices fixed) along a direction of at most 1 per logit: what a
    step h leaves is h^2 / 6 of a third derivative, at most 8 for a softmax
    whose logits move by at most 1; the values' own errors go by 1 / 2 h."""
    T, E, k, h = 64, 24, 4, 2.0 ** -7
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.round(64 * torch.randn(T, E, device="cuda", generator=g)) / 64
    ids, w0 = tg.moe_route(logits, k)
    step = torch.round(16 * (2 * torch.rand(T, E, device="cuda", generator=g) - 1)) / 16
    loss, counts, slope = tg.moe_balance(logits, ids)
    one = torch.ones((), device="cuda")
    d = tg.moe_route_backward(logits, ids, None, torch.empty_like(logits), slope=slope, dloss=one)
    up, down = (tg.moe_balance(logits + s * h * step, ids)[0].double() for s in (1, -1))
    err = lu.balance64(logits, ids, 1.0)[3] + 2.0 ** -22
    largest = float(counts.max()) * E / float(counts.sum())
    assert abs(float((up - down) / (2 * h)) - float((d * step).double().sum())) <= largest * 8 * h * h / 6 + err / h + 1e-6
    # the weights: choices that stay the same under the step
    gaps = logits.topk(k + 1, 1).values
    same = (gaps[:, :-1] - gaps[:, 1:]).min(1).values > 4 * h
    assert int(same.sum()) > T // 2
    dw = torch.rand(T, k, device="cuda", generator=g)
    for renormalize in (True, False):
        d = tg.moe_route_backward(logits, ids, dw, torch.empty_like(logits), renormalize=renormalize, scale=3.0)
        ends = [tg.moe_route(logits + s * h * step, k, renormalize=renormalize, scale=3.0) for s in (1, -1)]
        assert torch.equal(ends[0][0][same], ids[same]) and torch.equal(ends[1][0][same], ids[same])
        diff = ((ends[0][1] - ends[1][1]).double() * dw).sum(1) / (2 * h)
        off = (diff - (d * step).double().sum(1)).abs()[same]
        assert (off <= 3.0 * k * (8 * h * h / 6 + 80 * 2.0 ** -24 / h)).all()


@pytest.mark.parametrize("T", [50, 3000])
def test_streams_graphs_and_repeats(T):
    logits, ids, g = case(T, 64, 4, "f32")
    dw = torch.randn(T, 4, device="cuda", generator=g)
    run = lambda **kw: tg.moe_balance(logits, ids, **kw)  # noqa: E731
    want = run()
    one = torch.ones((), device="cuda")
    dl = gradient(logits, ids, dw, slope=want[2], dloss=one)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(stream=s)
    with torch.cuda.stream(s):
        d2 = torch.empty_like(logits)
    tg.moe_route_backward(logits, ids, dw, d2, slope=got[2], dloss=one, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(d2, dl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
        d3 = tg.moe_route_backward(logits, ids, dw, torch.zeros_like(logits), slope=out[2], dloss=one)
    for _ in range(3):
        logits.mul_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = run()
        assert all(torch.equal(a, b) for a, b in zip(out, now))
        assert torch.equal(d3, gradient(logits, ids, dw, slope=now[2], dloss=one))


def test_refusals_on_the_gpu():
    logits, ids, _ = case(20, 16, 2, "bf16")
    dw, slope, one = torch.zeros(20, 2, device="cuda"), torch.zeros(16, device="cuda"), torch.ones((), device="cuda")
    d = torch.empty_like(logits)
    before = tg.dispatch_count()
    back = tg.moe_route_backward
    bad = [lambda: tg.moe_balance(logits, ids.long()), lambda: tg.moe_balance(logits, ids[:10]),
           lambda: tg.moe_balance(logits, ids, coef=math.inf), lambda: tg.moe_balance(logits[0], ids),
           lambda: tg.moe_balance(logits, ids.cpu()), lambda: tg.moe_balance(logits[:0], ids[:0]),
           lambda: tg.moe_balance(logits[:, :1], ids), lambda: tg.moe_balance(logits[:1].expand(20, 16), ids),
           lambda: tg.moe_balance(logits, ids.repeat(1, 9)[:, :17].contiguous()),
           lambda: back(logits, ids, None, d), lambda: back(logits, ids, dw, d, slope=slope),
           lambda: back(logits, ids, dw, d, dloss=one), lambda: back(logits, ids, dw[:, :1], d),
           lambda: back(logits, ids, dw.half(), d), lambda: back(logits, ids, dw, d.half()),
           lambda: back(logits, ids, dw, d[:, :8]), lambda: back(logits, ids, dw, logits),
           lambda: back(logits, ids, dw, d, slope=slope[:8], dloss=one),
           lambda: back(logits, ids, dw, d, slope=slope, dloss=slope),
           lambda: back(logits, ids, dw, d, scale=math.nan)]
    for i, call in enumerate(bad):
        with pytest.raises(tg.TcGemmError):
            call()
            pytest.fail("call %d was not refused" % i)
    assert tg.dispatch_count() == before


@pytest.mark.parametrize("E", [8, 17, 64, 200, 512])
@pytest.mark.parametrize("ahead", [0, 1])
def test_around_one_workgroup(E, ahead):
    """As many tokens as one workgroup takes without scratch memory, and one
    more; logits that can and cannot be read 4 at a time."""
    most = 4 * 1024 // (16 if E <= 16 else 32 if E <= 32 else 64)
    for T in (most, most + 1):
        logits, ids, g = case(T, E, 2, "f32", seed=T + E)
        room = torch.zeros(T * E + 1, device="cuda")
        there = room[ahead:ahead + T * E].view(T, E)
        there.copy_(logits)
        balance(there, ids)


@pytest.mark.parametrize("E,k", [(2, 2), (16, 16), (60, 5), (64, 8), (200, 7), (256, 8), (500, 16), (512, 3)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_the_same_expert_again(E, k, renormalize):
    """Ids drawn with repetition from a few experts, and rows of one alone: the
    shares of the places add up."""
    T = 301
    logits, _, g = case(T, E, k, "f32")
    ids = torch.randint(0, max(2, min(E, 4)), (T, k), device="cuda", generator=g, dtype=torch.int32)
    ids[::5] = E - 1
    ids[::7, 0] = -1
    dw = torch.randn(T, k, device="cuda", generator=g)
    balance(logits, ids)
    gradient(logits, ids, dw, renormalize, 1.5, torch.randn(E, device="cuda"), torch.ones((), device="cuda"))
