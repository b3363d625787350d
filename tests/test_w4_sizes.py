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


# ------------------------------------------------------------------ sizes past 32 bits
def meta(shape, stride, dtype=torch.bfloat16):
    """A tensor without memory (only its sizes are looked at)."""
    return torch.empty_strided(shape, stride, dtype=dtype, device="meta")


BIG = 2 ** 32 + 256        # 256 once its upper bits are lost


def meta_weight(N, K):
    w = weight((), N, K)
    return tuple(t if t is None else t.to("meta") for t in w)


CALLS = [
    ("ldx", lambda: tg._make_qgemm(meta((2, 256), (BIG, 1)), meta_weight(64, 256), meta((2, 64), (64, 1)), 1, 0)),
    ("ldy", lambda: tg._make_qgemm(meta((2, 256), (256, 1)), meta_weight(64, 256), meta((2, 64), (BIG, 1)), 1, 0)),
    ("M", lambda: tg._make_qgemm(meta((BIG, 256), (256, 1)), meta_weight(64, 256), meta((BIG, 64), (64, 1)), 1, 0)),
    ("route ld", lambda: tg._make_route(meta((2, 64), (BIG, 1)), 2, True, 1.0)),
    ("route T", lambda: tg._make_route(meta((BIG, 64), (64, 1)), 2, True, 1.0)),
    ("top_k", lambda: tg._make_route(meta((2, 64), (64, 1)), 2 ** 32 + 2, True, 1.0)),
    ("layer ldy", lambda: tg._make_moe(meta((2, 64), (64, 1)), meta((2, 4), (4, 1)), meta((4, 2, 32, 64), (4096, 2048, 64, 1)),
                                       meta((4, 64, 32), (2048, 32, 1)), meta((2, 64), (BIG, 1)), 2, "silu", True,
                                       1.0, None)),
    ("layer ldx", lambda: tg._make_moe(meta((2, 64), (BIG, 1)), meta((2, 4), (4, 1)), meta((4, 2, 32, 64), (4096, 2048, 64, 1)),
                                       meta((4, 64, 32), (2048, 32, 1)), meta((2, 64), (64, 1)), 2, "silu", True,
                                       1.0, None)),
    ("matrices", lambda: tg._make_quantize(meta((2 ** 32 + 1, 16, 128), (2048, 128, 1)), 128, False, None)),
    ("rows", lambda: tg._make_quantize(meta((2 ** 32 + 16, 128), (128, 1)), 128, False, None)),
    ("columns", lambda: tg._make_quantize(meta((16, 2 ** 32 + 128), (2 ** 32 + 128, 1)), 128, False, None)),
    ("dequantized rows", lambda: tg._w4_desc((torch.empty(2 ** 28 + 1, 1, 1024, dtype=torch.uint8, device="meta"),
                                              torch.empty(2 ** 28 + 1, 1, 16, 1, dtype=torch.float16, device="meta"),
                                              None), 2 ** 32 + 16, 128)),
    ("dense lda", lambda: tg.make_desc(meta((2, 64), (BIG, 1)), meta((64, 8), (8, 1)), meta((2, 8), (8, 1)))),
    ("dense ldc", lambda: tg.make_desc(meta((2, 64), (64, 1)), meta((64, 8), (8, 1)), meta((2, 8), (BIG, 1)))),
    ("dense M", lambda: tg.make_desc(meta((BIG, 64), (64, 1)), meta((64, 8), (8, 1)), meta((BIG, 8), (8, 1)))),
    ("dense batch", lambda: tg.make_desc(meta((BIG, 2, 64), (128, 64, 1)), meta((64, 8), (8, 1)),
                                         meta((BIG, 2, 8), (16, 8, 1)))),
]


@pytest.mark.parametrize("name,call", CALLS, ids=[c[0] for c in CALLS])
def test_sizes_past_32_bits_are_refused(name, call):
    """A descriptor's 32-bit field would keep the lower half of such a size,
    and the call would read or write other rows than the tensor's."""
    with pytest.raises(tg.TcGemmError) as e:
        call()
    assert e.value.status == 3
