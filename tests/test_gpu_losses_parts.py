"""Gradients whose tokens are taken in parts: rows of x or of dx that span 2^31
elements and more (loss_util has the bounds)."""
import pytest
import torch

import loss_util as lu
import dense_gemm_tiled_amd as tg
from test_gpu_cross_entropy import backward, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [200, 700])
@pytest.mark.parametrize("dtype,dw,beta", [("f32", "own", 0.0), ("f32", "own", 0.5), ("bf16", "own", 0.0),
                                           ("bf16", "own", 0.5), ("bf16", "f32", 0.5), ("f16", "own", 1.0),
                                           ("f16", "f32", 0.0), ("bf16", None, 0.0)])
def test_rows_of_dx_far_apart(dtype, dw, beta, V):
    """An f32 dx of 1100 rows of 8 MiB."""
    T, H, ld = 1100, 64, 2097120
    assert (T - 1) * ld >= 2 ** 31
    x, w, targets, g = case(T, V, H, dtype, seed=V)
    old = torch.randn(V, H, device="cuda", generator=g)
    grad = torch.rand(T, device="cuda", generator=g) + 0.1
    dx, _ = backward(x, w, targets, grad, scale=0.5, dx="f32", dw=dw, beta=beta, old=old, pads=(ld - H, 3))
    assert (dx[~lu.counted(targets, V)] == 0).all()


@pytest.mark.parametrize("dtype,V,H,dx,dw,beta", [("bf16", 9000, 16384, "own", "own", 0.5), ("bf16", 300, 16383, "own", "own", 0.0),
                                                  ("f16", 300, 16384, "own", "f32", 1.0), ("f16", 300, 16384, None, "own", 0.0),
                                                  ("bf16", 300, 16384, "f32", "f32", 0.0), ("f32", 300, 16384, "own", "own", 1.0)])
def test_many_tokens(dtype, V, H, dx, dw, beta):
    """131300 tokens of 16384 numbers, one in 97 of which adds something; the
    last ones do."""
    T, scale = 131300, 1.0
    assert T * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(V + H)
    w = torch.empty(V, H, dtype=lu.DT[dtype], device="cuda").normal_(0.0, 2.0 / H ** 0.5, generator=g)
    x = torch.empty(T, H, dtype=lu.DT[dtype], device="cuda").normal_(generator=g)
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    t = torch.arange(T, device="cuda")
    keep = (t % 97 == 5) | (t >= T - 3)
    keep[65790:65794] = True
    targets[~keep & (t % 2 == 0)] = -100
    grad = torch.where(keep, torch.rand(T, device="cuda", generator=g) + 0.1, 0.0)
    xk, tk = x[keep], targets[keep]
    loss, lse = tg.cross_entropy(x, w, targets)
    want = lu.loss64(xk, w, tk, scale)
    lu.check(loss[keep], want[0], want[2], None, "f32", "loss")
    lu.check(lse[keep], want[1], want[3], None, "f32", "lse")
    own = lambda kind: lu.DT[dtype if kind == "own" else kind]  # noqa: E731
    outs = {"dx": None if dx is None else torch.full((T, H), float("nan"), dtype=own(dx), device="cuda"),
            "dw": torch.randn(V, H, device="cuda", generator=g).to(own(dw))}
    old = outs["dw"].clone()
    tg.cross_entropy_backward(x, w, targets, lse, grad, outs["dx"], outs["dw"], beta=beta)
    name = lambda kind: None if kind is None else dtype if kind == "own" else kind  # noqa: E731
    want = lu.grads64(xk, w, tk, lse[keep], grad[keep], scale, dtype, name(dx), name(dw), old, beta)
    if dx is not None:
        lu.check(outs["dx"][keep], *want["dx"], name(dx), "dx")
        assert (outs["dx"][~keep] == 0).all()
    lu.check(outs["dw"], *want["dw"], name(dw), "dw")


def test_the_same_bits_every_time():
    T, V, H, ld = 1100, 300, 64, 2097120
    x, w, targets, g = case(T, V, H, "bf16")
    grad = torch.rand(T, device="cuda", generator=g)
    lse = tg.cross_entropy(x, w, targets)[1]
    whole, first = torch.empty(T, ld, device="cuda"), None
    for _ in range(3):
        dx, dw = tg.cross_entropy_backward(x, w, targets, lse, grad, whole[:, :H], torch.empty_like(w))
        now = dx.clone(), dw
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


@pytest.mark.parametrize("rest", [1, 5, 20])
@pytest.mark.parametrize("dtype,dw", [("f32", "own"), ("bf16", "own"), ("f16", "f32")])
def test_few_tokens_in_the_last_part(dtype, dw, rest):
    """Four parts of 1024 tokens, and one of a few."""
    T, V, H, ld = 4096 + rest, 130, 40, 2097120
    x, w, targets, g = case(T, V, H, dtype, seed=rest)
    targets[-rest:] = torch.arange(rest, device="cuda") % V
    old = torch.randn(V, H, device="cuda", generator=g)
    grad = torch.rand(T, device="cuda", generator=g) + 0.1
    backward(x, w, targets, grad, dx="f32", dw=dw, beta=0.5, old=old, pads=(ld - H, 0))


def test_captured():
    """Tokens in parts in a graph, replayed after other work."""
    T, V, H, ld = 1100, 300, 64, 2097120
    x, w, targets, g = case(T, V, H, "bf16")
    grad = torch.rand(T, device="cuda", generator=g)
    lse = tg.cross_entropy(x, w, targets)[1]
    dx, dw = torch.zeros(T, ld, device="cuda")[:, :H], torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tg.cross_entropy_backward(x, w, targets, lse, grad, dx, dw)
    for n in range(3):
        grad.mul_(0.75)
        dx.fill_(0)
        dw.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = dx.clone(), dw.clone()
        tg.cross_entropy_backward(x, w, targets, lse, grad, dx, dw)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw), n
