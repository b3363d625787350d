"""The references of the 4-bit weight and mixture-of-experts tests, against
closed forms and against themselves (CPU)."""
import numpy as np
import pytest
import torch

import op_util as ou


def test_block_position_is_a_bijection():
    seen = {(b, s) for b, s in (ou.block_position(k) for k in range(128))}
    assert len(seen) == 128
    assert {b for b, _ in seen} == {kq * 256 + i * 4 + b for kq in range(4) for i in range(4)
                                    for b in range(4)}
    # the documented nibbles of one dword
    assert [ou.block_position(j) for j in range(8)] == [(0, 0), (2, 0), (0, 4), (2, 4), (1, 0),
                                                        (3, 0), (1, 4), (3, 4)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_random_weights_read_back(dtype, group, zeros):
    gen = torch.Generator().manual_seed(3)
    w = ou.w4_random(gen, (), 21, 150, dtype, group, zeros, "cpu")
    q, z, s = ou.w4_parts(w, 21, 150)
    assert q.min() == 0 and q.max() == 15 and np.isfinite(s).all()
    assert (z == 8).all() != zeros
    c = w[0].numpy()
    # row 17, column 130 = block (1, 1), row 1, k = 2: byte 16, high nibble
    assert q[17, 130] == c[1, 1, 16] >> 4


def test_quantize_ref_closed_forms():
    w = torch.zeros(5, 32)
    w[1] = 1.0                       # m = 1: s = -1/8, q = 8 - 8
    w[2, 3] = -4.0                   # m = -4: s = 0.5, q = 8 - 8 there
    w[3, :2] = torch.tensor([8.0, 1.5])     # s = -1: 1.5 / -1 is a tie, to even -2
    w[4, 0] = float("inf")
    q, z, s = ou.quantize_ref(w, 32, False, "f16")
    assert (q[0] == 8).all() and s[0] == 0
    assert (q[1] == 0).all() and s[1] == -0.125
    assert q[2, 3] == 0 and q[2, 0] == 8 and s[2] == 0.5
    assert q[3, 0] == 0 and q[3, 1] == 6 and s[3] == -1
    assert torch.isnan(s[4]).all()
    q, z, s = ou.quantize_ref(w[:4] - 1.0, 32, True, "bf16")
    assert (z[0] == 15).all() and (q[0] == 0).all()


def test_route_ref_ties_and_masks():
    l = torch.tensor([[1.0, 1.0, 1.0, 0.0], [float("-inf"), float("nan"), 2.0, float("-inf")],
                      [float("-inf")] * 4, [float("inf"), 1.0, float("inf"), 0.0]])
    ids, w = ou.route_ref(l, 2)
    assert ids.tolist() == [[0, 1], [2, -1], [-1, -1], [0, 2]]
    assert np.allclose(w, [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5]])


def test_gate_rejects_a_wrong_code():
    """The bound of the product passes an fp32 evaluation and rejects one
    whose weight differs by one step in one place."""
    gen = torch.Generator().manual_seed(4)
    N, K = 16, 256
    w = ou.w4_random(gen, (), N, K, "bf16", 128, False, "cpu")
    x = torch.randn(3, K, generator=gen).to(torch.bfloat16)
    v, b = ou.gemm_ref(x, w, N)
    d = torch.from_numpy(ou.w4_values(w, N, K))
    ou.check((x.float() @ d.float().T), v, b)
    d[5, 7] += d.abs().max() / 8
    with pytest.raises(AssertionError):
        ou.check((x.float() @ d.float().T), v, b)
