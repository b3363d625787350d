"""What a weight held in 4 bits knows of its matrices' sizes (host)."""
import copy
import pickle

import pytest
import torch

import dense_gemm_tiled_amd as tg


def weight(lead, N, K, sized=True):
    nb, kb = -(-N // 16), -(-K // 128)
    arrays = (torch.zeros(*lead, nb, kb, 1024, dtype=torch.uint8),
              torch.zeros(*lead, nb, kb, 16, 1, dtype=torch.bfloat16))
    return tg.W4Weight(*arrays, N=N, K=K) if sized else tg.W4Weight(*arrays)


def test_a_weight_is_its_three_arrays():
    w = weight((2,), 33, 40)
    codes, scales, zeros = w
    assert w.codes is codes and w.scales is scales and zeros is None and len(w) == 3
    assert (w.N, w.K) == (33, 40)
    for other in (copy.copy(w), pickle.loads(pickle.dumps(w))):
        assert (other.N, other.K) == (33, 40) and torch.equal(other.codes, codes)
    plain = weight((2,), 33, 40, sized=False)
    assert plain.N is None and plain.K is None and tg._as_w4(plain) == tuple(plain)


def test_intermediate_size_of_the_experts():
    up, dn = weight((4, 2), 33, 64), weight((4,), 64, 33)
    assert tg._intermediate(up, dn) == 33
    assert tg._intermediate(tuple(up), dn) == tg._intermediate(up, tuple(dn)) == 33
    assert tg._intermediate(tuple(up), tuple(dn)) is None
    with pytest.raises(tg.TcGemmError, match="33 rows and down 34"):
        tg._intermediate(up, weight((4,), 64, 34))
    with pytest.raises(tg.TcGemmError, match="33 rows and down 34"):
        tg.moe(torch.zeros(3, 64), torch.zeros(3, 4), up, weight((4,), 64, 34), torch.zeros(3, 64), top_k=2)


def test_the_size_reaches_the_layer():
    """The descriptor's I, with and without sizes and with one given."""
    x, y, route = torch.zeros(3, 64).bfloat16(), torch.zeros(3, 64), torch.zeros(3, 4)
    up, dn = weight((4, 2), 33, 64), weight((4,), 64, 33)

    def size(intermediate):
        return tg._make_moe(x, route, tuple(up), tuple(dn), y, 2, "silu", True, 1.0, intermediate)[0].I

    assert size(tg._intermediate(up, dn)) == 33
    assert size(None) == 48 and size(40) == 40
