"""The cross entropy and its gradients where rows are not whole 16-byte pieces:
few tokens read W in place, more copy it, a piece at a time (loss_util has the
bounds)."""
import pytest
import torch

import dense_gemm_tiled_amd as tg
import loss_util as lu
from test_gpu_cross_entropy import backward, case, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 4, 17, 64, 65, 128, 129, 256, 257, 300])
@pytest.mark.parametrize("V,H", [(700, 77), (33000, 131)])
def test_odd_rows(T, V, H, dtype):
    x, w, targets, g = case(T, V, H, dtype, seed=T)
    forward(x, w, targets)
    grad = torch.rand(T, device="cuda", generator=g) + 0.1
    backward(x, w, targets, grad)
    backward(x, w, targets, grad, dx=None)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [9, 64, 100, 200])
@pytest.mark.parametrize("pad", [(0, 3), (5, 0), (1, 1), (8, 7), (3, 8)])
def test_one_side(T, pad, dtype):
    """Whole pieces in each row, but rows that do not start on them (NaN in
    between)."""
    x, w, targets, g = case(T, 1500, 136, dtype, pad=pad)
    forward(x, w, targets)
    grad = torch.rand(T, device="cuda", generator=g) + 0.1
    backward(x, w, targets, grad, pads=(3, 1))
    backward(x, w, targets, grad, dx=None, dw="f32")
    backward(x, w, targets, grad, dx="f32", dw="f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [2, 64, 130, 300])
def test_infinite_rows(T, dtype):
    """A word whose row holds infinities next to one that is all but certain:
    the row beside it is not touched by them."""
    V, H = 500, 61
    x, w, targets, g = case(T, V, H, dtype)
    x = x.abs().clamp(min=0.125)
    w[100:104] = -float("inf")
    targets[(targets >= 100) & (targets < 104)] = 5
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[100:104] = False
    moved = torch.cumsum(keep, 0) - 1
    t2 = torch.where(targets >= 0, moved[targets.clamp(min=0)], targets)
    want, lse64, off, lse_off = lu.loss64(x, w[keep], t2)
    loss, lse = tg.cross_entropy(x, w, targets)
    lu.check(lse, lse64, lse_off, None, "f32", "lse")
    lu.check(loss, want, off, None, "f32", "loss")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [130, 260])
def test_pieces_of_copied_words(T, dtype):
    """More words than a piece of the copy holds (2^28 elements of whole rows)."""
    V, H = 70001, 4095
    x, w, targets, g = case(T, V, H, dtype)
    targets[:4] = torch.tensor([0, 65535, 65536, 70000], device="cuda")
    forward(x, w, targets)
    backward(x, w, targets, torch.rand(T, device="cuda", generator=g) + 0.1)


def test_captured():
    """Copies and products in a graph, replayed."""
    x, w, targets, g = case(200, 900, 75, "bf16")
    grad = torch.rand(200, device="cuda", generator=g)
    want = tg.cross_entropy(x, w, targets)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    tg.cross_entropy_backward(x, w, targets, want[1], grad, dx, dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dx2, dw2 = torch.empty_like(x), torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = tg.cross_entropy(x, w, targets)
        tg.cross_entropy_backward(x, w, targets, got[1], grad, dx2, dw2)
    for _ in range(3):
        dx2.fill_(0)
        dw2.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((got[0], want[0]), (got[1], want[1]), (dx2, dx), (dw2, dw)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("beta", [0.0, 0.5])
@pytest.mark.parametrize("T", [1, 4, 5, 8, 9, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("V,H", [(1, 1), (63, 255), (64, 256), (65, 257), (20011, 64), (70000, 300), (300, 5000)])
def test_few_tokens_in_fp32(V, H, T, beta):
    """Shares of words that end inside a wave's, columns that end inside one."""
    x, w, targets, g = case(T, V, H, "f32", seed=T + V, pad=(3, 1))
    old = torch.randn(V, H, device="cuda", generator=g)
    grad = torch.rand(T, device="cuda", generator=g) + 0.1
    backward(x, w, targets, grad, scale=-0.5, beta=beta, old=old, pads=(2, 5))


def test_few_tokens_in_fp32_over_pieces():
    """More words than a piece holds: dx goes on from the sums before."""
    T, V, H = 3, (1 << 20) + 65, 5
    x, w, targets, g = case(T, V, H, "f32")
    targets[:] = torch.tensor([0, 1 << 20, V - 1], device="cuda")
    backward(x, w, targets, torch.rand(T, device="cuda", generator=g) + 0.1)
