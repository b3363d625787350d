"""What the products and layers keep of a result's bits, on the GPU."""
import numpy as np
import pytest
import torch

import op_util as ou
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    import dense_gemm_tiled_amd as t
    t.load_library()
    return t


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("T,E,H,I", [(1, 2, 200, 200), (1, 2, 2064, 330), (3, 2, 72, 130), (5, 1, 72, 130),
                                     (6, 1, 300, 257), (40, 2, 100, 136), (140, 2, 40, 40)])
def test_layer_keeps_the_bits_of_h(tg, dtype, act, T, E, H, I):
    """f32 results hold act(gate) * up to f32's own accuracy (few tokens, the
    pairs of an expert in one pass and in several, and many).  Every x has
    one nonzero, so gate and up are single exact products, and down is the
    identity: y[n] = h[n].  h may be off by the activation's 16 u (of its
    argument, |g| <= 8 here) and its product with up, u; its parts add 2^-24 of it
    (bf16: 3 parts of 8 bits) or 2^-22 + 2^-25 (f16: two of 11, and half its
    smallest number).  Two bf16 parts are up to 2^-16 off."""
    gen = torch.Generator().manual_seed(T + H)
    n = min(H, I)
    x = torch.zeros(T, H)
    col = torch.randint(0, H, (T,), generator=gen)
    x[torch.arange(T), col] = torch.rand(T, generator=gen) + 0.5
    x = x.to(ou.DT[dtype])
    up = (torch.randn(E, 2, I, H, generator=gen)).clamp(-4, 4).to(ou.DT[dtype])
    dn = torch.zeros(E, H, I)
    dn[:, torch.arange(n), torch.arange(n)] = 1.0
    ids = torch.randint(0, E, (T, 1), generator=gen, dtype=torch.int32)
    y = torch.empty(T, H, device="cuda")
    say("GPU case: moe parts of h", T, E, H, I, dtype, act)
    tg.moe(x.cuda(), (ids.cuda(), torch.ones(T, 1, device="cuda")), up.cuda(), dn.to(ou.DT[dtype]).cuda(), y,
           activation=act)
    xs, w = ou.f64(x)[np.arange(T), col], ou.f64(up)[ids[:, 0].numpy()]
    g, u = (xs[:, None] * w[np.arange(T), s, :, col] for s in (0, 1))
    h = ou.act64(g, act) * u
    parts = 2.0 ** -24 * np.abs(h) if dtype == "bf16" else 2.0 ** -22 * np.abs(h) + 2.0 ** -25
    bound = np.zeros((T, H))
    bound[:, :n] = (np.abs(u) * 16 * ou.U * np.abs(g) + ou.U * np.abs(h) + parts)[:, :n]
    value = np.zeros((T, H))
    value[:, :n] = h[:, :n]
    ou.check(y, value, bound, "moe")
