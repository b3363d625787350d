"""The cross entropy of a linear layer and its gradients against 64 bits
(loss_util has the bounds)."""
import math

import pytest
import torch

import dense_gemm_tiled_amd as tg
import loss_util as lu

pytestmark = pytest.mark.gpu


def case(T, V, H, dtype, seed=1, scale=1.0, ignored=0.2, index=torch.int64, spread=2.5, boost=4.0, pad=(0, 0)):
    """x, w, targets: logits of about `spread`, the target's up to `boost`
    above; rows pad[0], pad[1] elements further apart than they are long."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w = (rnd(V, H) * (spread / math.sqrt(H) / abs(scale))).to(lu.DT[dtype])
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    rows = w[targets].float()
    up = boost * torch.rand(T, 1, device="cuda", generator=g) / (rows * rows).sum(1, keepdim=True).clamp(min=1e-3) / scale
    x = (rnd(T, H) + up * rows).to(lu.DT[dtype])
    targets[torch.rand(T, device="cuda", generator=g) < ignored] = -100

    def padded(t, n):
        if n == 0:
            return t
        whole = torch.full((t.size(0), t.size(1) + n), float("nan"), dtype=t.dtype, device="cuda")
        whole[:, :t.size(1)] = t
        return whole[:, :t.size(1)]
    return padded(x, pad[0]), padded(w, pad[1]), targets.to(index), g


def forward(x, w, targets, scale=1.0, **kw):
    loss, lse = tg.cross_entropy(x, w, targets, scale=scale, **kw)
    want, lse64, off, lse_off = lu.loss64(x, w, targets, scale)
    lu.check(lse, lse64, lse_off, None, "f32", "lse")
    lu.check(loss, want, off, None, "f32", "loss")
    assert (loss[~lu.counted(targets, w.size(0))] == 0).all()
    return loss, lse


def backward(x, w, targets, grad, scale=1.0, dx="own", dw="own", beta=0.0, lse=None, old=None, pads=(0, 0), **kw):
    own = lu.NAME[x.dtype]
    kinds = {"dx": own if dx == "own" else dx, "dw": own if dw == "own" else dw}
    if lse is None:
        live = lu.counted(targets, w.size(0))
        clean = torch.where(live[:, None], x, torch.zeros((), dtype=x.dtype, device="cuda"))
        lse = lu.loss64(clean, w, targets, scale)[1].float()
    outs, whole = {}, {}
    for (name, like), pad in zip((("dx", x), ("dw", w)), pads):
        if kinds[name] is None:
            outs[name] = None
            continue
        t = torch.full((like.size(0), like.size(1) + pad), float("nan"), dtype=lu.DT[kinds[name]], device="cuda")
        whole[name], outs[name] = t, t[:, :like.size(1)]
    if beta != 0.0:
        outs["dw"].copy_(old)
    before = None if beta == 0.0 else outs["dw"].clone()
    got = tg.cross_entropy_backward(x, w, targets, lse, grad, outs["dx"], outs["dw"], scale=scale, beta=beta, **kw)
    assert got[0] is outs["dx"] and got[1] is outs["dw"]
    torch.cuda.synchronize()
    want = lu.grads64(x, w, targets, lse, grad, scale, own, kinds["dx"], kinds["dw"], before, beta)
    for name, (value, each, var) in want.items():
        lu.check(outs[name], value, each, var, kinds[name], name)
        rest = whole[name][:, outs[name].size(1):]
        assert torch.isnan(rest).all(), "%s: written past its rows" % name
    return outs["dx"], outs["dw"]


SHAPES = [(1, 1, 1), (1, 2, 8), (2, 1, 16), (1, 257, 64), (3, 128, 72), (16, 300, 128), (17, 1000, 64),
          (64, 4099, 192), (129, 513, 136), (256, 256, 64), (257, 769, 520), (300, 4099, 1032),
          (5, 300, 7), (64, 1025, 100), (33, 129, 65), (1021, 5003, 264),
          (7, 130, 2056), (32, 65, 40), (31, 1000, 72), (300, 33101, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_loss(T, V, H, dtype):
    x, w, targets, _ = case(T, V, H, dtype, seed=T + V)
    forward(x, w, targets)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_gradients(T, V, H, dtype):
    x, w, targets, g = case(T, V, H, dtype, seed=T + V + 1)
    grad = (0.5 + torch.rand(T, device="cuda", generator=g)) / T * (1024 if dtype == "f16" else 1)
    backward(x, w, targets, grad)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [0.5, -1.0, -0.125, 3.0])
def test_scale(dtype, scale):
    x, w, targets, g = case(70, 400, 96, dtype, scale=scale)
    forward(x, w, targets, scale)
    backward(x, w, targets, torch.rand(70, device="cuda", generator=g), scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("beta", [0.0, 1.0])
@pytest.mark.parametrize("T,V,H,pad", [(1, 65, 8, 0), (31, 1000, 1032, 0), (32, 130, 136, 8), (33, 63, 2056, 3),
                                       (64, 5000, 72, 0), (50, 30000, 200, 5), (65, 700, 520, 0),
                                       (128, 1025, 264, 8), (100, 9000, 1288, 0)])
def test_gradients_of_few_tokens(T, V, H, pad, beta, dtype):
    x, w, targets, g = case(T, V, H, dtype, seed=T + V + 2)
    old = torch.randn(V, H, device="cuda", generator=g)
    backward(x, w, targets, torch.rand(T, device="cuda", generator=g) + 0.1, beta=beta, old=old, pads=(pad, pad))
    backward(x, w, targets, torch.rand(T, device="cuda", generator=g) + 0.1, dx=None, beta=beta, old=old)


@pytest.mark.parametrize("T,V,H,dtype", [(33000, 17000, 64, "bf16"), (5000, 20000, 16, "f32"),
                                         (4100, 40003, 24, "f16"), (4100, 40003, 23, "bf16")])
def test_many_pieces(T, V, H, dtype):
    """More tokens than a pass takes, more words than a piece holds."""
    x, w, targets, g = case(T, V, H, dtype)
    forward(x, w, targets)
    if T * V * 8 < 2 ** 31:
        backward(x, w, targets, torch.full((T,), 1.0 / T, device="cuda"))
    else:
        # (in 64 bits a part of the tokens at a time)
        grad = torch.where(torch.arange(T, device="cuda") % 7 == 0, 1.0, 0.0)
        keep = grad != 0
        lse = torch.zeros(T, device="cuda")
        lse[keep] = lu.loss64(x[keep], w, targets[keep])[1].float()
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        tg.cross_entropy_backward(x, w, targets, lse, grad, dx, dw)
        want = lu.grads64(x[keep], w, targets[keep], lse[keep], grad[keep], 1.0, dtype, dtype, dtype)
        lu.check(dx[keep], *want["dx"], dtype, "dx")
        lu.check(dw, *want["dw"], dtype, "dw")
        assert (dx[~keep] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,V,H", [(9, 200, 64), (130, 700, 136), (40, 300, 33)])
@pytest.mark.parametrize("dx,dw", [("f32", "f32"), ("own", "f32"), ("f32", "own"), (None, "f32"), ("f32", None)])
def test_f32_gradients(dtype, T, V, H, dx, dw):
    x, w, targets, g = case(T, V, H, dtype)
    backward(x, w, targets, torch.rand(T, device="cuda", generator=g), dx=dx, dw=dw)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dx,dw", [(None, "own"), ("own", None)])
def test_one_gradient(dtype, dx, dw):
    x, w, targets, g = case(50, 333, 88, dtype)
    backward(x, w, targets, torch.rand(50, device="cuda", generator=g), dx=dx, dw=dw)


@pytest.mark.parametrize("dtype,dw", [("bf16", "own"), ("bf16", "f32"), ("f16", "own"), ("f16", "f32"), ("f32", "own")])
@pytest.mark.parametrize("beta", [1.0, -0.5])
def test_beta(dtype, dw, beta):
    x, w, targets, g = case(150, 500, 136, dtype)
    old = torch.randn(500, 136, device="cuda", generator=g)
    backward(x, w, targets, torch.rand(150, device="cuda", generator=g), dw=dw, beta=beta, old=old)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [8, 3])
def test_pitches(dtype, pad):
    """Rows further apart than they are long: what lies between is neither
    read (NaN) nor written."""
    x, w, targets, g = case(140, 600, 128, dtype, pad=(pad, pad))
    forward(x, w, targets)
    backward(x, w, targets, torch.rand(140, device="cuda", generator=g), pads=(pad, pad))
    backward(x, w, targets, torch.rand(140, device="cuda", generator=g), dx="f32", dw="f32", pads=(pad, pad))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_odd_addresses(dtype):
    x, w, targets, g = case(130, 300, 64, dtype)
    flat = torch.empty(300 * 64 + 1, dtype=w.dtype, device="cuda")
    w1 = flat[1:].view(300, 64).copy_(w)
    flat = torch.empty(130 * 64 + 1, dtype=x.dtype, device="cuda")
    x1 = flat[1:].view(130, 64).copy_(x)
    grad = torch.rand(130, device="cuda", generator=g)
    for a, b in ((x1, w), (x, w1), (x1, w1)):
        forward(a, b, targets)
        backward(a, b, targets, grad)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_targets_outside(dtype, index):
    x, w, targets, g = case(12, 260, 64, dtype, ignored=0.0, index=index)
    last = 2 ** 31 - 1
    outside = [260, -1, -100, last, -2 ** 31] + ([2 ** 40 + 5, -2 ** 40, 2 ** 32] if index is torch.int64 else [261, -2, last - 1])
    targets[:8] = torch.tensor(outside, dtype=index, device="cuda")
    targets[8:] = torch.tensor([0, 259, 128, 127], dtype=index, device="cuda")
    loss, _ = forward(x, w, targets)
    assert (loss[:8] == 0).all() and (loss[8:] > 0).all()
    dx, _ = backward(x, w, targets, torch.rand(12, device="cuda", generator=g) + 0.5)
    assert (dx[:8] == 0).all() and (dx[8:] != 0).any(1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H", [64, 61])
def test_ignored_tokens_may_hold_anything(dtype, H):
    x, w, targets, g = case(100, 300, H, dtype, ignored=0.5)
    live = lu.counted(targets, 300)
    grad = torch.rand(100, device="cuda", generator=g) + 0.5
    dx0, dw0 = backward(x, w, targets, grad)
    lse = tg.cross_entropy(x, w, targets)[1]
    x1, grad1, lse1 = x.clone(), grad.clone(), lse.clone()
    x1[~live] = float("nan")
    x1[~live, ::3] = float("inf")
    grad1[~live] = float("nan")
    lse1[~live] = float("nan")
    loss, l1 = tg.cross_entropy(x1, w, targets)
    assert torch.equal(loss, tg.cross_entropy(x, w, targets)[0]) and torch.equal(l1[live], lse[live])
    a = tg.cross_entropy_backward(x, w, targets, lse, grad, torch.empty_like(x), torch.empty_like(w))
    b = tg.cross_entropy_backward(x1, w, targets, lse1, grad1, torch.empty_like(x), torch.empty_like(w))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (b[0][~live] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_all_ignored(dtype):
    x, w, targets, _ = case(40, 300, 64, dtype, ignored=1.1)
    loss, lse = forward(x, w, targets)
    assert (loss == 0).all() and torch.isfinite(lse).all()
    old = torch.randn(300, 64, device="cuda").to(w.dtype)
    dw = old.clone()
    dx, dw = tg.cross_entropy_backward(x, w, targets, lse, torch.ones(40, device="cuda"),
                                       torch.full_like(x, float("nan")), dw, beta=1.0)
    assert (dx == 0).all() and torch.equal(dw, old)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_nan_and_infinity_stay_with_their_token(dtype):
    x, w, targets, _ = case(300, 400, 64, dtype, ignored=0.0)
    want = tg.cross_entropy(x, w, targets)
    x = x.clone()
    x[7, 3] = float("nan")
    x[133, 5] = float("inf")
    loss, lse = tg.cross_entropy(x, w, targets)
    rest = torch.ones(300, dtype=torch.bool, device="cuda")
    rest[[7, 133]] = False
    assert torch.isnan(loss[7]) and torch.isnan(lse[7])
    assert not torch.isfinite(lse[133])
    assert torch.equal(loss[rest], want[0][rest]) and torch.equal(lse[rest], want[1][rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("big", [60.0, 3e4])
def test_far_logits(dtype, big):
    """Products far from 0, most of them far below the largest: losses of all
    but certain tokens near 0, of surprised ones as large as the products."""
    H, V, T = 64, 700, 90
    w = torch.zeros(V, H, device="cuda")
    w[torch.arange(V), torch.arange(V) % H] = 1.0
    w = w * torch.linspace(0.5, 1.0, V, device="cuda")[:, None]
    x = torch.zeros(T, H, device="cuda")
    x[torch.arange(T), torch.arange(T) % H] = big
    x, w = x.to(lu.DT[dtype]), w.to(lu.DT[dtype])
    targets = torch.arange(T, device="cuda") % H + 640 - 64 * (torch.arange(T, device="cuda") % 2)
    targets = torch.where(targets < V, targets, 5)
    forward(x, w, targets)
    forward(x, w, targets, -1.0)
    backward(x, w, targets, torch.ones(T, device="cuda"))


def test_certain_tokens_have_small_losses():
    """A loss is as exact as its products also where lse and the target's
    product agree to all but a few bits, and so is the target's gradient."""
    T, V, H = 64, 512, 64
    w = torch.zeros(V, H, device="cuda", dtype=torch.bfloat16)
    w[:H] = torch.eye(H, device="cuda").to(w.dtype)
    x = torch.eye(H, device="cuda").to(w.dtype)[:T] * 16
    targets = torch.arange(T, device="cuda")
    loss, lse = tg.cross_entropy(x, w, targets)
    want = math.log1p((V - 1) * math.exp(-16.0))
    # (512 exponentials, their sum and its logarithm: 1 + 5.75e-5 in steps of 2^-23)
    assert (loss.double() - want).abs().max() <= 2.0 ** -22
    dx, dw = tg.cross_entropy_backward(x, w, targets, lse, torch.ones(T, device="cuda"), torch.empty_like(x),
                                       torch.empty(V, H, device="cuda"))
    p = math.exp(16.0 - float(lse[0]))
    got = dx.diagonal().double()
    # expm1(16 - lse), lse rounded to 2^-20: within 2^-20 of p - 1 = -5.75e-5, then bf16
    assert (got - (p - 1)).abs().max() <= 2.0 ** -20 + 2.0 ** -8 * (1 - p)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_grad_forms(dtype):
    """One number for all tokens, an expanded one, every second of a longer
    tensor, zeros among them."""
    x, w, targets, g = case(64, 300, 64, dtype)
    one = torch.full((), 0.25, device="cuda")
    a = backward(x, w, targets, one)
    b = backward(x, w, targets, one.expand(64))
    c = backward(x, w, targets, torch.full((1,), 0.25, device="cuda"))
    d = backward(x, w, targets, torch.full((64,), 0.25, device="cuda"))
    for other in (b, c, d):
        assert torch.equal(a[0], other[0]) and torch.equal(a[1], other[1])
    long = torch.rand(128, device="cuda", generator=g)
    long[::8] = 0.0
    dx, _ = backward(x, w, targets, long[::2])
    assert (dx[::4] == 0).all()


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e12])
def test_grad_sizes(size):
    """f16 gradients are scaled by the largest grad: tiny and huge ones lose
    nothing.  Results in f32, which hold them."""
    x, w, targets, g = case(64, 300, 64, "f16")
    grad = (torch.rand(64, device="cuda", generator=g) + 0.5) * size
    backward(x, w, targets, grad, dx="f32", dw="f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_gradient_against_differences(dtype):
    """Central differences of the framework's own losses along a direction:
    with products moving by at most a along it, the third derivative of lse is
    at most (2 a)^3, a step h leaves h^2 / 6 of it, and the losses' own
    errors are divided by 2 h."""
    T, V, H, h = 24, 150, 64, 2.0 ** -8
    x, w, targets, g = case(T, V, H, "f32", ignored=0.25)
    x, w = x.to(lu.DT[dtype]).float(), w.to(lu.DT[dtype]).float()
    loss, lse = tg.cross_entropy(x, w, targets)
    grad = torch.rand(T, device="cuda", generator=g)
    dx, dw = tg.cross_entropy_backward(x.to(lu.DT[dtype]), w.to(lu.DT[dtype]), targets, lse, grad,
                                       torch.empty_like(x), torch.empty_like(w))
    for which in ("x", "w"):
        d = torch.randn(x.shape if which == "x" else w.shape, device="cuda", generator=g)
        d = torch.round(d * 16) / 16
        ends, errs = [], []
        for sign in (1, -1):
            a, b = (x + sign * h * d, w) if which == "x" else (x, w + sign * h * d)
            ends.append(tg.cross_entropy(a, b, targets)[0].double())
            errs.append(lu.loss64(a, b, targets)[2])
        slope = float((grad.double() * (ends[0] - ends[1])).sum()) / (2 * h)
        move = (d.double() @ w.double().t()) if which == "x" else (x.double() @ d.double().t())
        a3 = (2 * move.abs().max(1).values) ** 3
        c = lu.counted(targets, V)
        room = float((grad.double() * c * (a3 * h * h / 6 + (errs[0] + errs[1]) / (2 * h))).sum())
        got = float(((dx if which == "x" else dw).double() * d.double()).sum())
        want = lu.grads64(x, w, targets, lse, grad, 1.0, dtype, "f32", "f32")["dx" if which == "x" else "dw"]
        room += float((want[1] * d.abs().double()).sum())
        assert abs(got - slope) <= room, (which, got, slope, room)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,H", [(1, 4096, 256), (200, 3001, 128)])
def test_same_bits_every_time(dtype, T, V, H):
    x, w, targets, g = case(T, V, H, dtype)
    grad = torch.rand(T, device="cuda", generator=g)
    first = None
    for _ in range(3):
        loss, lse = tg.cross_entropy(x, w, targets)
        dx, dw = tg.cross_entropy_backward(x, w, targets, lse, grad, torch.empty_like(x), torch.empty_like(w))
        now = [loss, lse, dx, dw]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_captured_and_replayed(dtype):
    """Two graphs of the same calls on two streams, replayed side by side,
    with other work between the replays."""
    data = [case(130, 900, 128, dtype, seed=s) for s in (1, 2)]
    grad = torch.rand(130, device="cuda", generator=data[0][3])
    graphs, outs = [], []
    tg.cross_entropy(*data[0][:3])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (x, w, t, _), s in zip(data, streams):
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            loss, lse = tg.cross_entropy(x, w, t)
            dx, dw = tg.cross_entropy_backward(x, w, t, lse, grad, torch.zeros_like(x), torch.zeros_like(w))
        graphs.append(graph)
        outs.append((loss, lse, dx, dw))
    for n in range(4):
        for x, w, t, _ in data:
            x.mul_(0.9)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (x, w, t, _), got in zip(data, outs):
            loss, lse = tg.cross_entropy(x, w, t)
            dx, dw = tg.cross_entropy_backward(x, w, t, lse, grad, torch.empty_like(x), torch.empty_like(w))
            for a, b in zip(got, (loss, lse, dx, dw)):
                assert torch.equal(a, b), n


def test_other_stream():
    x, w, targets, g = case(100, 5000, 256, "bf16")
    grad = torch.rand(100, device="cuda", generator=g)
    loss, lse = tg.cross_entropy(x, w, targets)
    dx, dw = tg.cross_entropy_backward(x, w, targets, lse, grad, torch.empty_like(x), torch.empty_like(w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    loss2, lse2 = tg.cross_entropy(x, w, targets, stream=s)
    with torch.cuda.stream(s):
        dx2, dw2 = torch.empty_like(x), torch.empty_like(w)
    tg.cross_entropy_backward(x, w, targets, lse2, grad, dx2, dw2, stream=s)
    s.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_armed_measurement_waits_for_a_gemm():
    x, w, targets, _ = case(70, 300, 61, "bf16")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(), b.record()
    torch.cuda.synchronize()
    tg.time_next_gemm(a, b)
    forward(x, w, targets)
    c = torch.empty(64, 64, device="cuda")
    tg.gemm(torch.ones(64, 64, device="cuda"), torch.ones(64, 64, device="cuda"), c)
    torch.cuda.synchronize()
    assert a.elapsed_time(b) >= 0 and (c == 64).all()


def test_refusals_on_the_gpu():
    x, w, targets, g = case(20, 100, 64, "bf16")
    before = tg.dispatch_count()
    loss, lse = torch.zeros(20, device="cuda"), torch.zeros(20, device="cuda")
    grad = torch.ones(20, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    bad = [lambda: tg.cross_entropy(x, w.float(), targets), lambda: tg.cross_entropy(x, w[:, :32], targets),
           lambda: tg.cross_entropy(x, w, targets[:10]), lambda: tg.cross_entropy(x, w, targets.float()),
           lambda: tg.cross_entropy(x, w, targets, scale=0.0), lambda: tg.cross_entropy(x, w, targets, scale=math.inf),
           lambda: tg.cross_entropy(x[0], w, targets), lambda: tg.cross_entropy(x.cpu(), w, targets),
           lambda: tg.cross_entropy(x[:0], w, targets[:0]), lambda: tg.cross_entropy(x.to(torch.int8), w, targets),
           lambda: tg.cross_entropy(x[:1].expand(20, 64), w, targets),
           lambda: tg.cross_entropy(x.t().contiguous().t(), w, targets),
           lambda: tg.cross_entropy_backward(x, w, targets, lse, grad),
           lambda: tg.cross_entropy_backward(x, w, targets, lse[:5], grad, dx),
           lambda: tg.cross_entropy_backward(x, w, targets, lse, grad[:5], dx),
           lambda: tg.cross_entropy_backward(x, w, targets, lse, grad.double(), dx),
           lambda: tg.cross_entropy_backward(x, w, targets, lse, grad, dx[:, :8]),
           lambda: tg.cross_entropy_backward(x, w, targets, lse, grad, dx.half()),
           lambda: tg.cross_entropy_backward(x, w, targets, lse, grad, dx, dw, beta=math.nan),
           lambda: tg.cross_entropy_backward(x, w, targets, lse, grad, x),
           lambda: tg.cross_entropy_backward(x, w, targets, lse, grad, dx, w)]
    for i, call in enumerate(bad):
        with pytest.raises(tg.TcGemmError):
            call()
            pytest.fail("call %d was not refused" % i)
    assert tg.dispatch_count() == before
