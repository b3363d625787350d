"""The losses' products leave an armed measurement to the next GEMM call."""
import pytest
import torch

import dense_gemm_tiled_amd as tg
from test_gpu_cross_entropy import backward, case, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,H,dtype", [(70, 300, 61, "bf16"), (2, 300, 61, "bf16"), (200, 900, 64, "bf16"), (9, 500, 64, "f32")])
def test_events_are_recorded_around_the_gemm_and_not_before(T, V, H, dtype):
    """Events that a product inside a loss had taken would lie before one that is
    recorded behind the losses."""
    x, w, targets, g = case(T, V, H, dtype)
    start, end, behind = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    start.record(), end.record()
    torch.cuda.synchronize()
    tg.time_next_gemm(start, end)
    forward(x, w, targets)
    backward(x, w, targets, torch.rand(T, device="cuda", generator=g) + 0.1)
    a, c = torch.ones(64, 64, device="cuda"), torch.empty(64, 64, device="cuda")
    behind.record()
    tg.gemm(a, a, c)
    torch.cuda.synchronize()
    assert behind.elapsed_time(start) >= 0 and start.elapsed_time(end) > 0 and (c == 64).all()
