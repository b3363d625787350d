"""The losses' operators from several threads and streams at once: every result
is that of the call alone, to the bit."""
import threading

import pytest
import torch

import dense_gemm_tiled_amd as tg
from test_gpu_cross_entropy import case

pytestmark = pytest.mark.gpu

SIZES = [(1, 9000, 256, "bf16"), (60, 5000, 512, "f16"), (300, 3001, 136, "bf16"), (40, 2000, 77, "bf16"),
         (9, 4000, 64, "f32"), (200, 3000, 100, "f32")]


def step(x, w, targets, grad, logits, k, stream):
    loss, lse = tg.cross_entropy(x, w, targets, stream=stream)
    with torch.cuda.stream(stream):
        dx, dw, dl = torch.empty_like(x), torch.empty_like(w), torch.empty_like(logits)
    tg.cross_entropy_backward(x, w, targets, lse, grad, dx, dw, stream=stream)
    with torch.cuda.stream(stream):
        ids, weights = tg.moe_route(logits, k)
    balance, counts, slope = tg.moe_balance(logits, ids, stream=stream)
    tg.moe_route_backward(logits, ids, weights, dl, slope=slope, dloss=balance, stream=stream)
    return loss, lse, dx, dw, balance, counts, slope, dl


def test_threads_and_streams():
    data = []
    for i, (T, V, H, dtype) in enumerate(SIZES):
        x, w, targets, g = case(T, V, H, dtype, seed=i)
        data.append((x, w, targets, torch.rand(T, device="cuda", generator=g),
                     torch.randn(50 * T, 64, device="cuda", generator=g), 4))
    main = torch.cuda.current_stream()
    want = [step(*d, main) for d in data]
    torch.cuda.synchronize()
    results, errors = [[] for _ in data], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(5):
                results[i].append(step(*data[i], s))
            s.synchronize()
        except Exception as e:                      # (shown below, in the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for i, runs in enumerate(results):
        assert len(runs) == 5
        for run in runs:
            for a, b in zip(run, want[i]):
                assert torch.equal(a, b), i
