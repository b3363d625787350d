"""Cases of the 4-bit weight and mixture-of-experts operators, with their plain forms.

Operators: ``w4_quantize`` (with ``w4_dequantize``: a weight matrix through the
4-bit format and back), ``w4_gemm`` (y = act(x @ W^T + bias), W held in 4
bits with group scales), ``moe_route`` (the top_k experts of each token and
their softmax weights) and ``moe`` (a whole mixture-of-experts layer, experts
held in 16 or 4 bits).

The 4-bit format, as the framework documents it: a block is 16 rows x 128
values of K in 1024 bytes, [4 (kq), 16 (row), 4 (i), 4 bytes]; the four bytes
of (kq, row, i) hold k = 32 i + 8 kq + j, j = 0..7, in nibbles: byte 0 holds
j = 0 (low) and 2 (high), byte 1 j = 4 and 6, byte 2 j = 1 and 3, byte 3
j = 5 and 7.  codes [.., ceil(N/16), ceil(K/128), 1024] uint8, scales and
zeros [.., ceil(N/16), ceil(K/128), 16, 128/G].  W = scale * (code - zero),
zero 8 where none is held.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases
def _gemm(name, M, N, K, dtype, group, zeros, bias=False, act="none", out=None):
    return {"name": name, "op": "w4_gemm", "M": M, "N": N, "K": K, "dtype": dtype, "group": group,
            "zeros": zeros, "bias": bias, "act": act, "out": out or dtype}


def _moe(name, T, H, I, E, k, dtype, held, group=128, zeros=False, renorm=True, act="silu"):
    return {"name": name, "op": "moe", "T": T, "H": H, "I": I, "E": E, "k": k, "dtype": dtype,
            "held": held, "group": group, "zeros": zeros, "renorm": renorm, "act": act}


def listed():
    return [
        # one token through a square projection: the smallest call, latency counts
        _gemm("w4_gemm_token", 1, 4096, 4096, "bf16", 128, False),
        # a few sequences decoding through a wide projection
        _gemm("w4_gemm_decode", 4, 16384, 8192, "f16", 128, False),
        # odd sizes, a short last group, zero points, bias and activation in the epilogue
        _gemm("w4_gemm_ragged", 13, 4099, 4093, "bf16", 32, True, bias=True, act="gelu_tanh"),
        # a batch of 64 decoding sequences, fp32 results
        _gemm("w4_gemm_batch", 64, 8192, 4096, "bf16", 64, True, out="f32"),
        # a prompt
        _gemm("w4_gemm_prompt", 2048, 4096, 4096, "bf16", 128, False),
        # a bf16 checkpoint's matrix into the 4-bit format
        {"name": "w4_quantize_bf16", "op": "w4_quantize", "N": 8192, "K": 4096, "wdtype": "bf16",
         "dtype": "bf16", "group": 128, "zeros": False},
        # fp32 master weights of odd sizes, zero points
        {"name": "w4_quantize_f32", "op": "w4_quantize", "N": 4099, "K": 4093, "wdtype": "f32",
         "dtype": "f16", "group": 32, "zeros": True},
        # one decoding token's routing
        {"name": "moe_route_token", "op": "moe_route", "T": 1, "E": 128, "k": 8, "dtype": "f32",
         "renorm": True},
        # a prompt's routing: bf16 logits (ties), some experts masked for some tokens
        {"name": "moe_route_prompt", "op": "moe_route", "T": 4096, "E": 256, "k": 8, "dtype": "bf16",
         "renorm": False},
        # one decoding token, 16-bit experts
        _moe("moe_token", 1, 2048, 1024, 64, 8, "bf16", "dense"),
        # a small decoding batch, 4-bit experts
        _moe("moe_w4_batch", 16, 4096, 1408, 64, 8, "bf16", "w4"),
        # a larger batch of odd size, fp16 experts, odd intermediate size
        _moe("moe_batch", 61, 4096, 1400, 32, 4, "f16", "dense", renorm=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4_gemm", "w4_gemm", "w4_quantize", "moe_route", "moe", "moe"])
    dtype = rng.choice(["bf16", "f16"])
    group, zeros = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "w4_gemm":
        M = _log(rng, 1, 512)
        N, K = _log(rng, 256, 8192), _log(rng, 256, 8192)
        if rng.random() < 0.5:
            N, K = N // 16 * 16, K // 128 * 128
        c = _gemm("", M, N, K, dtype, group, zeros, rng.random() < 0.5,
                  rng.choice(["none", "relu", "gelu_tanh"]), rng.choice([dtype, "f32"]))
    elif op == "w4_quantize":
        c = {"op": op, "N": _log(rng, 64, 8192), "K": _log(rng, 128, 4096),
             "wdtype": rng.choice(["f32", "f16", "bf16"]), "dtype": dtype, "group": group,
             "zeros": zeros}
    elif op == "moe_route":
        E = rng.randint(8, 256)
        c = {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, 8),
             "dtype": rng.choice(["f32", "f16", "bf16"]), "renorm": rng.random() < 0.5}
    else:
        E = rng.choice([8, 16, 24, 60, 64])
        c = _moe("", _log(rng, 1, 128), rng.randint(8, 32) * 64, rng.randint(64, 1024), E,
                 rng.randint(1, min(8, E)), dtype, rng.choice(["dense", "w4"]), group, zeros,
                 rng.random() < 0.5, rng.choice(["silu", "gelu_tanh"]))
    c.pop("name", None)
    return c


# ------------------------------------------------------------------ inputs
def _w4_inputs(lead, N, K, dtype, group, zeros, g):
    """Random codes (bell-shaped, as quantized weights are), scales and zero
    points of `lead` matrices [N, K]; the products' outputs are of order 1."""
    nb, kb = (N + 15) // 16, (K + 127) // 128
    r1 = torch.randint(0, 256, (*lead, nb, kb, 1024), dtype=torch.uint8, device="cuda", generator=g)
    r2 = torch.randint(0, 256, (*lead, nb, kb, 1024), dtype=torch.uint8, device="cuda", generator=g)
    lo, hi = ((r1 & 15) + (r2 & 15) + 1) >> 1, ((r1 >> 4) + (r2 >> 4) + 1) >> 1
    codes = lo | (hi << 4)
    shape = (*lead, nb, kb, 16, 128 // group)
    s = torch.rand(shape, device="cuda", generator=g) + 0.5
    s = s * torch.where(torch.rand(shape, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    s = (s * (0.3 / math.sqrt(K))).to(_DT[dtype])
    z = torch.randint(5, 12, shape, dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    return codes, s, z


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype="f32", scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(_DT[dtype])

    c, st = case, {"case": case}
    if c["op"] == "w4_gemm":
        st["x"] = randn(c["M"], c["K"], dtype=c["dtype"])
        st["w"] = _w4_inputs((), c["N"], c["K"], c["dtype"], c["group"], c["zeros"], g)
        st["bias"] = randn(c["N"], dtype=c["out"]) if c["bias"] else None
        st["y"] = torch.empty(c["M"], c["N"], dtype=_DT[c["out"]], device="cuda")
    elif c["op"] == "w4_quantize":
        st["w"] = randn(c["N"], c["K"], dtype=c["wdtype"], scale=1 / math.sqrt(c["K"]))
        st["out"] = torch.empty(c["N"], c["K"], dtype=torch.float32, device="cuda")
    elif c["op"] == "moe_route":
        st["logits"] = randn(c["T"], c["E"], dtype=c["dtype"])
        gone = torch.rand(c["T"], c["E"], device="cuda", generator=g) < 0.1
        gone &= torch.rand(c["T"], 1, device="cuda", generator=g) < 0.3
        st["logits"].masked_fill_(gone, -math.inf)
    else:
        T, H, I, E = c["T"], c["H"], c["I"], c["E"]
        st["x"] = randn(T, H, dtype=c["dtype"])
        st["logits"] = randn(T, E)
        if c["held"] == "w4":
            st["gate_up"] = _w4_inputs((E, 2), I, H, c["dtype"], c["group"], c["zeros"], g)
            st["down"] = _w4_inputs((E,), H, I, c["dtype"], c["group"], c["zeros"], g)
        else:
            st["gate_up"] = torch.empty(E, 2, I, H, dtype=_DT[c["dtype"]], device="cuda")
            st["gate_up"].normal_(0.0, 1 / math.sqrt(H), generator=g)
            st["down"] = torch.empty(E, H, I, dtype=_DT[c["dtype"]], device="cuda")
            st["down"].normal_(0.0, 1 / math.sqrt(I), generator=g)
        st["y"] = torch.empty(T, H, dtype=_DT[c["dtype"]], device="cuda")
    return st


# ------------------------------------------------------------------ the framework's calls
def _run_own(st):
    import dense_gemm_tiled_amd as tg
    c = st["case"]
    if c["op"] == "w4_gemm":
        return tg.w4_gemm(st["x"], st["w"], st["y"], bias=st["bias"], activation=c["act"])
    if c["op"] == "w4_quantize":
        w4 = tg.w4_quantize(st["w"], group=c["group"], zeros=c["zeros"], scale_dtype=_DT[c["dtype"]])
        return tg.w4_dequantize(w4, st["out"])
    if c["op"] == "moe_route":
        return tg.moe_route(st["logits"], c["k"], renormalize=c["renorm"])
    return tg.moe(st["x"], st["logits"], st["gate_up"], st["down"], st["y"], top_k=c["k"],
                  activation=c["act"], renormalize=c["renorm"],
                  intermediate=c["I"])


# ------------------------------------------------------------------ plain forms
def _act(x, name):
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return torch.clamp(x, min=0) if name == "relu" else x


def _dense(w, N, K):
    """The matrices that (codes, scales, zeros) stand for, in fp32 [.., N, K]."""
    codes, scales, zeros = w
    lead = codes.shape[:-3]
    nb, kb = codes.shape[-3:-1]
    n = len(lead)
    b = codes.reshape(*lead, nb, kb, 4, 16, 4, 2, 2, 1)              # .. kq row i half byte nibble
    q = torch.cat([b & 15, b >> 4], dim=-1)
    ax = [n, n + 3, n + 1, n + 4, n + 2, n + 6, n + 7, n + 5]        # .. nb row kb i kq byte nibble half
    q = q.permute(*range(n), *ax).reshape(*lead, nb * 16, kb, scales.shape[-1], -1).float()

    def per_group(t):                                                # [.., nb, kb, 16, G'] -> rows
        return t.transpose(-3, -2).reshape(*lead, nb * 16, kb, -1, 1).float()

    z = 8.0 if zeros is None else per_group(zeros)
    return ((q - z) * per_group(scales)).reshape(*lead, nb * 16, kb * 128)[..., :N, :K]


def _route(logits, k, renorm):
    l = logits.float()
    top, ids = torch.sort(l, dim=-1, descending=True, stable=True)
    m = top[:, :1].clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(top - m)
    p = e[:, :k] / (e[:, :k] if renorm else e).sum(-1, keepdim=True).clamp(min=1e-30)
    gone = top[:, :k] == -math.inf
    return ids[:, :k].masked_fill(gone, -1).to(torch.int32), p.masked_fill(gone, 0.0)


def _plain(st):
    c = st["case"]
    if c["op"] == "w4_gemm":
        y = st["x"].float() @ _dense(st["w"], c["N"], c["K"]).t()
        if st["bias"] is not None:
            y = y + st["bias"].float()
        return _act(y, c["act"]).to(_DT[c["out"]])
    if c["op"] == "w4_quantize":
        N, K, G = c["N"], c["K"], c["group"]
        w = torch.nn.functional.pad(st["w"].float(), (0, -K % G)).reshape(N, -1, G)
        hi, lo = w.amax(-1, keepdim=True), w.amin(-1, keepdim=True)
        if c["zeros"]:
            hi, lo = hi.clamp(min=0), lo.clamp(max=0)
            s = ((hi - lo) / 15).to(_DT[c["dtype"]]).double()
            z = torch.round(-lo.double() / s).clamp(0, 15)
            q = (torch.round(w.double() / s) + z).clamp(0, 15) - z
        else:
            s = (torch.where(-lo > hi, lo, hi) / -8).to(_DT[c["dtype"]]).double()
            q = torch.round(w.double() / s).clamp(-8, 7)
        return torch.where(s == 0, 0.0, q * s).reshape(N, -1)[:, :K].float()
    if c["op"] == "moe_route":
        return _route(st["logits"], c["k"], c["renorm"])
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    ids, p = _route(st["logits"], k, c["renorm"])
    x, up, down = st["x"].float(), st["gate_up"], st["down"]
    if T * k <= E:
        # few choices: gather the chosen experts
        at = ids.flatten().long().clamp(min=0)
        if c["held"] == "w4":
            up = _dense([t if t is None else t[at] for t in up], I, H)
            down = _dense([t if t is None else t[at] for t in down], H, I)
        else:
            up, down = up[at].float(), down[at].float()
        gu = (up.reshape(T, k, 2 * I, H) @ x[:, None, :, None]).reshape(T, k, 2, I)
        h = _act(gu[:, :, 0], c["act"]) * gu[:, :, 1]
        y = (down.reshape(T, k, H, I) @ h[..., None])[..., 0]
        return (y * p[..., None]).sum(1).to(_DT[c["dtype"]])
    # every expert for every token, weighted by its routing weight (0 where not chosen)
    up = (_dense(up, I, H) if c["held"] == "w4" else up.float()).reshape(E * 2 * I, H)
    down = _dense(down, H, I) if c["held"] == "w4" else down.float()
    full = torch.zeros(T, E + 1, device=x.device).scatter_(1, (ids + 1).long(), p)[:, 1:]
    gu = (x @ up.t()).reshape(T, E, 2, I)
    h = _act(gu[:, :, 0], c["act"]) * gu[:, :, 1] * full[..., None]
    return (h.reshape(T, E * I) @ down.transpose(1, 2).reshape(E * I, H)).to(_DT[c["dtype"]])


def run(state):
    return _run_own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _exact_dense(w, N, K):
    """One matrix [N, K] of the format in fp64, element by element from the
    position of its nibble."""
    codes, scales, zeros = w
    n = torch.arange(N, device=codes.device)[:, None]
    k = torch.arange(K, device=codes.device)[None, :]
    i, kq, j = k % 128 // 32, k % 32 // 8, k % 8
    byte = (kq * 16 + n % 16) * 16 + i * 4 + (j % 2) * 2 + j // 4
    q = codes[n // 16, k // 128, byte].to(torch.int64) >> (j // 2 % 2 * 4) & 15
    g = k % 128 // (128 // scales.shape[-1])
    z = 8.0 if zeros is None else zeros[n // 16, k // 128, n % 16, g].double()
    return (q.double() - z) * scales[n // 16, k // 128, n % 16, g].double()


def _exact_route(logits, k, renorm):
    l = logits.double()
    T, E = l.shape
    before = torch.zeros(T, E, dtype=torch.int64, device=l.device)   # how many come before it
    for e in range(E):
        o = l[:, e:e + 1]
        before += (o > l) | ((o == l) & (torch.arange(E, device=l.device) > e))
    ids = torch.full((T, k), -1, dtype=torch.int32, device=l.device)
    p = torch.zeros(T, k, dtype=torch.float64, device=l.device)
    t, e = torch.nonzero((before < k) & (l > -math.inf), as_tuple=True)
    ids[t, before[t, e]] = e.to(torch.int32)
    m = torch.where(l.amax(1) > -math.inf, l.amax(1), 0.0)
    p[t, before[t, e]] = torch.exp(l[t, e] - m[t])
    total = p.sum(1) if renorm else torch.exp(l - m[:, None]).sum(1)
    return ids, torch.where(total[:, None] > 0, p / total[:, None], 0.0)


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "w4_gemm":
        y = torch.matmul(st["x"].double(), _exact_dense(st["w"], c["N"], c["K"]).t().contiguous())
        return _act(y if st["bias"] is None else y + st["bias"].double(), c["act"])
    if c["op"] == "w4_quantize":
        w, out = st["w"].double(), torch.empty(c["N"], c["K"], dtype=torch.float64, device="cuda")
        for k0 in range(0, c["K"], c["group"]):
            v = w[:, k0:k0 + c["group"]]
            hi, lo = v.max(1, keepdim=True).values, v.min(1, keepdim=True).values
            if c["zeros"]:
                hi, lo = torch.maximum(hi, 0 * hi), torch.minimum(lo, 0 * lo)
                s, least = (hi - lo) / 15, 0 * lo
            else:
                s, least = torch.where(hi >= -lo, hi, lo) / -8, 0 * lo - 8
            s = s.to(_DT[c["dtype"]]).double()                       # the format holds 16-bit scales
            d = torch.where(s == 0, 1.0, s)
            z = torch.clamp(torch.round(-lo / d), 0, 15) if c["zeros"] else 0 * lo
            q = torch.minimum(torch.maximum(torch.round(v / d) + z, least), least + 15) - z
            out[:, k0:k0 + c["group"]] = q * s
        return out
    if c["op"] == "moe_route":
        return _exact_route(st["logits"], c["k"], c["renorm"])
    I, H = c["I"], c["H"]
    ids, p = _exact_route(st["logits"], c["k"], c["renorm"])
    x, y = st["x"].double(), torch.zeros(c["T"], H, dtype=torch.float64, device="cuda")
    for e in torch.unique(ids[ids >= 0]).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if c["held"] == "w4":
            g, u = [_exact_dense([v if v is None else v[e, s] for v in st["gate_up"]], I, H) for s in (0, 1)]
            d = _exact_dense([v if v is None else v[e] for v in st["down"]], H, I)
        else:
            g, u, d = st["gate_up"][e, 0].double(), st["gate_up"][e, 1].double(), st["down"][e].double()
        h = _act(torch.matmul(x[t], g.t().contiguous()), c["act"]) * torch.matmul(x[t], u.t().contiguous())
        y.index_add_(0, t, torch.matmul(h, d.t().contiguous()) * p[t, j][:, None])
    return y


# ------------------------------------------------------------------ what a pass cannot do without
def _w4_bytes(N, K, group, zeros):
    return N * K / 2 + N * -(-K // group) * (3 if zeros else 2)


def work(case):
    c = case
    if c["op"] == "w4_gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": _w4_bytes(N, K, c["group"], c["zeros"]) + M * K * 2 + M * N * _ES[c["out"]]
                + (N * _ES[c["out"]] if c["bias"] else 0), "flops": 2.0 * M * N * K}
    if c["op"] == "w4_quantize":
        # the weights read, the 4-bit form written and read, the values written
        return {"bytes": c["N"] * c["K"] * (_ES[c["wdtype"]] + 4)
                + 2 * _w4_bytes(c["N"], c["K"], c["group"], c["zeros"]), "flops": 4.0 * c["N"] * c["K"]}
    if c["op"] == "moe_route":
        return {"bytes": c["T"] * (c["E"] * _ES[c["dtype"]] + c["k"] * 8), "flops": 4.0 * c["T"] * c["E"]}
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    used = E * (1 - (1 - k / E) ** T)                                # experts touched, on average
    if c["held"] == "w4":
        per = 2 * _w4_bytes(I, H, c["group"], c["zeros"]) + _w4_bytes(H, I, c["group"], c["zeros"])
    else:
        per = 6 * I * H
    return {"bytes": used * per + T * (4 * H + 4 * E), "flops": 6.0 * T * k * I * H}
