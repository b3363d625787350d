"""Routing and whole mixture-of-experts layers on the GPU, against the plain
64-bit forms within their bounds (op_util)."""
import numpy as np
import pytest
import torch

import op_util as ou
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = ou.DT
NINF = float("-inf")


@pytest.fixture(scope="module")
def tg():
    import dense_gemm_tiled_amd as t
    t.load_library()
    return t


def rand(gen, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(DT[dtype])


# ------------------------------------------------------------------ routing
def check_route(tg, logits, k, renorm=True, scale=1.0):
    say("GPU case: moe_route", tuple(logits.shape), logits.dtype, k, renorm)
    ids, w = tg.moe_route(logits.cuda(), k, renormalize=renorm, scale=scale)
    rid, rw = ou.route_ref(logits, k, renorm, scale)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), rid)
    # an exponential, a sum of at most 512 terms, a quotient, the scale
    assert (np.abs(ou.f64(w) - rw) <= (ou.gamma(16 + 10) + 8 * ou.U) * np.abs(rw) + 2.0 ** -140).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (3, 64, 6), (5, 65, 2), (9, 128, 16), (33, 200, 8),
                                   (70, 256, 4), (6, 512, 16)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(tg, dtype, T, E, k, renorm):
    gen = torch.Generator().manual_seed(T + E)
    check_route(tg, rand(gen, T, E, dtype=dtype, scale=2.0), k, renorm, scale=2.5)


def test_route_ties_masks_and_infinities(tg):
    gen = torch.Generator().manual_seed(2)
    l = torch.randint(-2, 3, (40, 96), generator=gen).float()    # ties everywhere, zeros among them
    l[0] = 0
    l[1] = NINF                                                   # nothing to choose
    l[2] = NINF
    l[2, 50] = -3.0
    l[3, ::2] = float("nan")
    l[4] = torch.finfo(torch.float32).min                         # the type's lowest value as a mask
    l[4, 7] = 1.0
    l[5] = torch.finfo(torch.float32).min
    l[6, 3], l[6, 90] = float("inf"), float("inf")
    l[7, ::3] = -0.0
    for renorm in (True, False):
        check_route(tg, l, 6, renorm)
    check_route(tg, l.half().clamp(min=-65504), 6)


def test_route_strided_rows(tg):
    gen = torch.Generator().manual_seed(3)
    store = rand(gen, 11, 77, dtype="bf16").cuda()
    ids, w = tg.moe_route(store[:, 3:43], 5)
    i2, w2 = tg.moe_route(store[:, 3:43].contiguous(), 5)
    assert torch.equal(ids, i2) and torch.equal(w, w2)


# ------------------------------------------------------------------ the layer
def experts(gen, E, H, I, dtype, held):
    """(gate_up, down, gate_up(e, s), down(e)): what the call takes, and the
    matrices one by one.  held: None or (group, zeros)."""
    if held is None:
        up, dn = rand(gen, E, 2, I, H, dtype=dtype, scale=H ** -0.5), rand(gen, E, H, I, dtype=dtype, scale=I ** -0.5)
        return up.cuda(), dn.cuda(), lambda e, s: up[e, s], lambda e: dn[e]
    up = ou.w4_random(gen, (E, 2), I, H, dtype, *held, "cuda")
    dn = ou.w4_random(gen, (E,), H, I, dtype, *held, "cuda")
    return (up, dn, lambda e, s: [t if t is None else t[e, s] for t in up],
            lambda e: [t if t is None else t[e] for t in dn])


def run_layer(tg, T, H, I, E, k, dtype, held, act="silu", renorm=True, out=None, seed=1, logits=None, pads=(0, 0)):
    out = out or dtype
    gen = torch.Generator().manual_seed(seed)
    x = torch.full((T, H + pads[0]), float("nan"), dtype=DT[dtype])
    x[:, :H] = rand(gen, T, H, dtype=dtype)
    l = rand(gen, T, E) if logits is None else logits
    up, dn, gu, d = experts(gen, E, H, I, dtype, held)
    ys = torch.full((T, H + pads[1]), 7.0, dtype=DT[out], device="cuda")
    y = ys[:, :H]
    say("GPU case: moe", T, H, I, E, k, dtype, held, act, out, pads)
    r = tg.moe(x.cuda()[:, :H], l.cuda(), up, dn, y, top_k=k, activation=act, renormalize=renorm, intermediate=I)
    assert r is y
    ids, w = ou.route_ref(l, k, renorm)
    v, e = ou.moe_ref(x[:, :H], ids, w, gu, d, I, act, out)
    ou.check(y, v, e, "moe")
    assert (ys[:, H:] == 7).all()


HELD = [None, (32, True), (64, False), (64, True), (128, False), (128, True), (32, False)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("T", [1, 2, 16, 19, 130])
def test_layer(tg, dtype, held, T):
    run_layer(tg, T, 160, 96, 12, 3, dtype, held, seed=T)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 1, 1, 1, 1), (1, 8, 3, 4, 4), (2, 17, 31, 5, 2), (4, 129, 127, 3, 1),
                                       (7, 130, 17, 70, 16), (33, 96, 130, 2, 2), (128, 40, 40, 3, 2),
                                       (129, 72, 24, 300, 8), (300, 48, 33, 5, 5), (3, 600, 257, 16, 8),
                                       (1, 520, 1030, 9, 8), (16, 300, 300, 512, 4)])
@pytest.mark.parametrize("dtype,held", [("bf16", None), ("f16", (32, True)), ("bf16", (128, False))])
def test_layer_ragged(tg, T, H, I, E, k, dtype, held):
    run_layer(tg, T, H, I, E, k, dtype, held, out="f32", renorm=False, seed=T + H)


@pytest.mark.parametrize("held", [None, (64, True)])
@pytest.mark.parametrize("T", [3, 40])
def test_layer_gelu_strides(tg, held, T):
    run_layer(tg, T, 100, 48, 6, 2, "f16", held, act="gelu_tanh", pads=(5, 9))


@pytest.mark.parametrize("held", [None, (128, False)])
@pytest.mark.parametrize("T", [20, 128, 150])
def test_every_token_to_one_expert(tg, held, T):
    """All rows of a chunk through one expert, the other experts empty."""
    l = torch.full((T, 8), NINF)
    l[:, 5] = 1.0
    l[:, 2] = torch.where(torch.arange(T) % 7 == 0, 0.5, NINF)
    run_layer(tg, T, 136, 64, 8, 2, "bf16", held, logits=l)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("held", [None, (128, False), (64, True), (32, True)])
@pytest.mark.parametrize("T", [9, 17, 128, 150])
def test_few_of_many_experts(tg, dtype, held, T):
    """Many experts, nearly all tokens to the same two: the kernels that are
    chosen for few pairs an expert go through their list in many passes."""
    l = rand(torch.Generator().manual_seed(T), T, 150)
    l[:, 7] += 30
    l[: T - 3, 149] += 20
    run_layer(tg, T, 140, 33, 150, 2, dtype, held, logits=l, seed=T)


@pytest.mark.parametrize("held,dtype", [(h, ("f16", "bf16")[i % 2]) for i, h in enumerate(HELD)])
@pytest.mark.parametrize("H,I,E,k", [(9, 130, 5, 3), (24, 385, 4, 2), (100, 128, 3, 3), (2048, 257, 4, 2),
                                     (2049, 200, 4, 2), (2500, 640, 9, 8)])
def test_one_token(tg, H, I, E, k, held, dtype):
    """Both widths of the second product, whole and odd numbers of blocks."""
    run_layer(tg, 1, H, I, E, k, dtype, held, out="f32", seed=H + I)


def test_tokens_without_experts(tg):
    """A padded batch: tokens whose mask leaves no expert get zeros, even
    where x is NaN; a batch of nothing but those too."""
    gen = torch.Generator().manual_seed(4)
    up, dn, gu, d = experts(gen, 6, 64, 32, "bf16", None)
    for T, empty in ((5, [1, 4]), (3, [0, 1, 2]), (140, list(range(100, 140)))):
        x, l = rand(gen, T, 64, dtype="bf16"), rand(gen, T, 6)
        x[empty], l[empty] = float("nan"), NINF
        y = torch.full((T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        tg.moe(x.cuda(), l.cuda(), up, dn, y, top_k=2)
        ids, w = ou.route_ref(l, 2)
        x[empty] = 0
        v, e = ou.moe_ref(x, ids, w, gu, d, 32, "silu", "bf16")
        ou.check(y, v, e)
        assert (y[empty] == 0).all()


@pytest.mark.parametrize("held", [None, (32, True)])
def test_ids_and_weights(tg, held):
    """The caller's own routing: ids outside the experts add nothing, an id
    named twice counts with the sum of its weights, weights of any sign."""
    gen = torch.Generator().manual_seed(5)
    T, H, I, E, k = 21, 96, 40, 10, 4
    up, dn, gu, d = experts(gen, E, H, I, "f16", held)
    x = rand(gen, T, H, dtype="f16")
    ids = torch.randint(0, E, (T, k), generator=gen, dtype=torch.int32)
    ids[0] = -1
    ids[1] = torch.tensor([3, 3, 3, 3])
    ids[2] = torch.tensor([E, 2, -7, 2])
    ids[3] = torch.tensor([2 ** 31 - 1, -2 ** 31, 1, 1 << 20])
    w = rand(gen, T, k)
    y = torch.full((T, H), 7.0, dtype=torch.float16, device="cuda")
    tg.moe(x.cuda(), (ids.cuda(), w.cuda()), up, dn, y, intermediate=I)
    inside = torch.where((ids < 0) | (ids >= E), -1, ids).numpy()
    v, e = ou.moe_ref(x, inside, ou.f64(w), gu, d, I, "silu", "f16")
    ou.check(y, v, e)
    assert (y[0] == 0).all()


def test_logits_and_their_ids_agree(tg):
    gen = torch.Generator().manual_seed(6)
    for T in (1, 30, 200):
        up, dn, _, _ = experts(gen, 16, 128, 64, "bf16", None)
        x, l = rand(gen, T, 128, dtype="bf16").cuda(), rand(gen, T, 16, dtype="bf16").cuda()
        a, b = (torch.empty(T, 128, dtype=torch.float32, device="cuda") for _ in range(2))
        tg.moe(x, l, up.view(16, 128, 128), dn, a, top_k=4, scale=1.5)
        tg.moe(x, tg.moe_route(l, 4, scale=1.5), up, dn, b)
        assert torch.equal(a, b)


def test_router_quantizer_and_layer_together(tg):
    """As they are used: the router's product, experts quantized once, the
    layer, then a 4-bit projection of its output, on a side stream."""
    gen = torch.Generator().manual_seed(7)
    T, H, I, E, k, V = 6, 256, 112, 8, 2, 300
    dense_up, dense_dn = rand(gen, E, 2, I, H, dtype="bf16", scale=H ** -0.5), rand(gen, E, H, I, dtype="bf16", scale=I ** -0.5)
    head, router = rand(gen, V, H, dtype="bf16", scale=H ** -0.5), rand(gen, E, H, dtype="bf16", scale=H ** -0.5)
    x = rand(gen, T, H, dtype="bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        xc = x.cuda()
        up, dn, wh = (tg.w4_quantize(t.cuda(), group=64, zeros=True) for t in (dense_up, dense_dn, head))
        logits = tg.gemm(xc, router.cuda(), torch.empty(T, E, device="cuda"), transpose_b=True)
        y = tg.moe(xc, logits, up, dn, torch.empty_like(xc), top_k=k, intermediate=I)
        z = tg.w4_gemm(y, wh, torch.empty(T, V, device="cuda"))
    s.synchronize()
    ids, w = ou.route_ref(logits, k)
    one = lambda t, *i: [v if v is None else v[i] for v in t]  # noqa: E731
    v, e = ou.moe_ref(x, ids, w, lambda a, b: one(up, a, b), lambda a: one(dn, a), I, "silu", "bf16")
    ou.check(y, v, e)
    v, e = ou.gemm_ref(y.cpu(), wh, V)
    ou.check(z, v, e)


def test_same_result_every_time(tg):
    gen = torch.Generator().manual_seed(8)
    for T in (1, 16, 128, 300):
        for held in (None, (128, False)):
            up, dn, _, _ = experts(gen, 8, 256, 128, "bf16", held)
            x, l = rand(gen, T, 256, dtype="bf16").cuda(), rand(gen, T, 8).cuda()
            ys = [tg.moe(x, l, up, dn, torch.empty(T, 256, device="cuda"), top_k=3) for _ in range(3)]
            assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("T", [1, 20])
def test_captured_and_replayed(tg, T):
    """Two graphs of the layer, each with its own scratch memory, replayed on
    two streams at once; eager calls between them."""
    gen = torch.Generator().manual_seed(9)
    E, H, I, k = 8, 192, 64, 2
    up, dn, _, _ = experts(gen, E, H, I, "f16", None)
    xs = [rand(gen, T, H, dtype="f16").cuda() for _ in range(2)]
    ls = [rand(gen, T, E).cuda() for _ in range(2)]
    ys = [torch.zeros(T, H, dtype=torch.float16, device="cuda") for _ in range(2)]
    tg.moe(xs[0], ls[0], up, dn, ys[0], top_k=k)
    graphs = []
    for x, l, y in zip(xs, ls, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tg.moe(x, l, up, dn, y, top_k=k)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for step in range(4):
        for x, l, y in zip(xs, ls, ys):
            x.copy_(rand(gen, T, H, dtype="f16"))
            l.copy_(rand(gen, T, E))
            y.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for x, l, y in zip(xs, ls, ys):
            assert torch.equal(y, tg.moe(x, l, up, dn, torch.empty_like(y), top_k=k)), step


def test_large_expert_offsets(tg):
    """Experts past 4 GiB of one tensor: the last one's results."""
    E, H, I, T = 260, 2048, 2048, 2
    up = torch.zeros(E, 2, I, H, dtype=torch.bfloat16, device="cuda")
    dn = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
    assert up.numel() * 2 > 2 ** 32
    gen = torch.Generator().manual_seed(10)
    up[E - 1], dn[E - 1] = rand(gen, 2, I, H, dtype="bf16", scale=H ** -0.5).cuda(), rand(gen, H, I, dtype="bf16", scale=I ** -0.5).cuda()
    x = rand(gen, T, H, dtype="bf16")
    ids = torch.tensor([[E - 1, 0], [3, E - 1]], dtype=torch.int32)
    w = torch.tensor([[0.75, 0.25], [0.5, 0.5]])
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    tg.moe(x.cuda(), (ids.cuda(), w.cuda()), up, dn, y)
    g, d = up[E - 1].cpu(), dn[E - 1].cpu()
    only = np.where(ids.numpy() == E - 1, 0, -1)
    v, e = ou.moe_ref(x, only, ou.f64(w), lambda _, s: g[s], lambda _: d, I, "silu", "bf16")
    ou.check(y, v, e)


def test_refusals_launch_nothing(tg):
    gen = torch.Generator().manual_seed(11)
    E, H, I = 4, 64, 32
    up, dn, _, _ = experts(gen, E, H, I, "bf16", None)
    qu, qd, _, _ = experts(gen, E, H, I, "bf16", (64, False))
    x, l = rand(gen, 3, H, dtype="bf16").cuda(), rand(gen, 3, E).cuda()
    y = torch.full((3, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ids, w = tg.moe_route(l, 2)
    n0 = tg.dispatch_count()
    call = lambda x=x, r=l, up=up, dn=dn, y=y, **kw: tg.moe(x, r, up, dn, y, **{"top_k": 2, **kw})  # noqa: E731
    bad = [lambda: call(top_k=None), lambda: call(top_k=5), lambda: call(top_k=0), lambda: call(activation="relu"),
           lambda: call(x=x.half()), lambda: call(x=x[:, :63]), lambda: call(y=y.half()), lambda: call(y=x),
           lambda: call(r=l[:2]), lambda: call(r=l[:, :3]), lambda: call(r=l.cpu()), lambda: call(r=l.to(torch.int8)),
           lambda: call(r=(ids.long(), w)), lambda: call(r=(ids, w.half())), lambda: call(r=(ids, w[:2])),
           lambda: call(r=(ids.t().contiguous().t(), w)), lambda: call(r=(ids, w), top_k=3), lambda: call(r=(ids,)),
           lambda: call(up=up[:, :, :16]), lambda: call(up=up.half()), lambda: call(dn=dn[:, :, :16]),
           lambda: call(dn=dn.transpose(1, 2)), lambda: call(up=qu), lambda: call(up=qu, dn=dn),
           lambda: call(up=qu, dn=(qd[0], qd[1][..., :1].contiguous())), lambda: call(up=qu, dn=qd, intermediate=33),
           lambda: call(intermediate=16), lambda: call(scale=float("nan")), lambda: call(x=x[:0], r=l[:0], y=y[:0]),
           lambda: tg.moe_route(l, 5), lambda: tg.moe_route(l, 0), lambda: tg.moe_route(l[0], 1),
           lambda: tg.moe_route(l.to(torch.int32), 1)]
    for i, f in enumerate(bad):
        with pytest.raises(tg.TcGemmError):
            f()
            pytest.fail("refusal %d" % i)
    assert tg.dispatch_count() == n0
    torch.cuda.synchronize()
    assert (y == 7).all()
