"""Cases of the losses that a step of training computes, with their plain forms.

Operators: ``cross_entropy`` (the softmax cross entropy of a linear layer over
a large vocabulary: loss and log-sum-exp of each token, no logits kept),
``cross_entropy_backward`` (its gradients with respect to the activations and
the weight), ``moe_balance`` (the balance loss of a router, the tokens of each
expert, and what its gradient needs) and ``moe_route_backward`` (the gradient
of the router's logits: through the weights that ``moe_route`` gave and
through the balance loss).

    l[t, v]  = scale <x[t], W[v]>,   lse[t] = log sum_v exp l[t, v]
    loss[t]  = lse[t] - l[t, target[t]], 0 where the target is outside [0, V)
    G[t, v]  = grad[t] (exp(l[t, v] - lse[t]) - [v = target[t]]), 0 there
    dx = scale G W,   dW = scale G^T x

    p = softmax(logits[t]); a token counts where one of its ids is inside [0, E)
    counts[e] = places of ids that hold e, total their sum, n tokens that count
    loss     = coef E sum_e counts[e] / total * (sum_t p[t, e]) / n
    slope[e] = coef (E counts[e] - total) / (total n)
    weights  = scale softmax(logits[t, ids[t]]), or scale p[t, ids[t]]
    dlogits  = (d weights / d logits)^T dweights + dloss p (slope - sum_e p[e] slope[e])
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases
def _ce(name, T, V, H, dtype, scale=1.0, ignored=0.1, back=False):
    return {"name": name, "op": "cross_entropy_backward" if back else "cross_entropy", "T": T, "V": V,
            "H": H, "dtype": dtype, "scale": scale, "ignored": ignored}


def _router(name, back, T, E, k, dtype, renorm=True, padded=0.1):
    return {"name": name, "op": "moe_route_backward" if back else "moe_balance", "T": T, "E": E, "k": k,
            "dtype": dtype, "renorm": renorm, "padded": padded}


def listed():
    return [
        # the score of one token: the smallest call, latency counts
        _ce("loss_token", 1, 32768, 2048, "bf16", ignored=0.0),
        # the last tokens of 64 sequences scored against a large vocabulary
        _ce("loss_batch", 64, 131072, 4096, "bf16", ignored=0.0),
        # odd numbers of tokens and words, a logit scale, a third of the tokens a prompt's (ignored)
        _ce("loss_ragged", 1021, 50021, 2056, "f16", scale=0.5, ignored=0.3),
        # a micro-batch of a training step
        _ce("loss_train", 4096, 131072, 4096, "bf16"),
        # gradients of a small fp32 model
        _ce("grad_f32", 255, 10007, 1024, "f32", back=True),
        # gradients of a few scored tokens over a large vocabulary
        _ce("grad_batch", 64, 65536, 4096, "bf16", ignored=0.0, back=True),
        # odd sizes, fp16 with a loss scale
        _ce("grad_ragged", 1021, 50021, 2056, "f16", scale=0.5, ignored=0.3, back=True),
        # a micro-batch of a training step
        _ce("grad_train", 4096, 131072, 4096, "bf16", back=True),
        # the router of a small model, a short sequence
        _router("balance_small", False, 61, 8, 2, "f32"),
        # a training step's router
        _router("balance_train", False, 32768, 256, 8, "f32"),
        # a short sequence of odd length, experts not a power of two, bf16 logits
        _router("route_grad_small", True, 1021, 60, 4, "bf16"),
        # a training step's router, weights over all experts
        _router("route_grad_train", True, 32768, 256, 8, "f32", renorm=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross_entropy", "cross_entropy_backward", "moe_balance", "moe_route_backward"])
    if op.startswith("cross"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        small = dtype == "f32"
        H = rng.randint(8, 128 if small else 512) * 8
        if rng.random() < 0.2:
            H -= rng.randint(1, 7)                   # rows that are not whole 16-byte pieces
        c = _ce("", _log(rng, 1, 512 if small else 4096), _log(rng, 256, 16384 if small else 65536), H, dtype,
                rng.choice([1.0, 1.0, 0.5, -0.25]), rng.choice([0.0, 0.1, 0.5]), op.endswith("backward"))
    else:
        E = rng.randint(4, 256)
        c = _router("", op.endswith("backward"), _log(rng, 1, 32768), E, rng.randint(1, min(8, E)),
                    rng.choice(["f32", "f16", "bf16"]), rng.random() < 0.5, rng.choice([0.0, 0.2]))
    c.pop("name", None)
    return c


# ------------------------------------------------------------------ inputs
def _cross_inputs(c, g):
    """Activations and a weight whose logits have a spread of about 2.5, the
    target's word above that by up to 0.8 log V: as trained models have it,
    some words are all but certain and most losses are of order 1 to 10."""
    T, V, H, dt = c["T"], c["V"], c["H"], _DT[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    w = torch.empty(V, H, dtype=dt, device="cuda").normal_(0.0, 2.5 / math.sqrt(H) / abs(c["scale"]), generator=g)
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    rows = w[targets].float()
    boost = 0.8 * math.log(V) * torch.rand(T, 1, device="cuda", generator=g) / (rows * rows).sum(1, keepdim=True) / c["scale"]
    x = (randn(T, H) + boost * rows).to(dt)
    targets[torch.rand(T, device="cuda", generator=g) < c["ignored"]] = -100
    return x, w, targets


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, st = case, {"case": case}
    if c["op"].startswith("cross"):
        st["x"], st["w"], st["targets"] = _cross_inputs(c, g)
        if c["op"].endswith("backward"):
            # what the forward pass left, and the gradient of a weighted mean (fp16: scaled by 1024)
            st["lse"] = torch.logsumexp(c["scale"] * (st["x"].float() @ st["w"].float().t()), 1)
            weight = 0.5 + torch.rand(c["T"], device="cuda", generator=g)
            st["grad"] = weight * ((1024.0 if c["dtype"] == "f16" else 1.0) / c["T"])
            st["dx"] = torch.empty_like(st["x"])
            st["dw"] = torch.empty_like(st["w"])
        return st
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn(T, E, device="cuda", generator=g) + 0.3 * torch.randn(E, device="cuda", generator=g)
    logits = logits.to(_DT[c["dtype"]])
    logits.masked_fill_(torch.rand(T, E, device="cuda", generator=g) < 0.01, -math.inf)
    top, ids = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    ids = ids[:, :k].to(torch.int32).masked_fill(top[:, :k] == -math.inf, -1)
    # padding: no expert, and nothing that counts in the logits
    pad = torch.rand(T, device="cuda", generator=g) < c["padded"]
    st["logits"] = logits.masked_fill(pad[:, None], math.nan)
    st["ids"] = ids.masked_fill(pad[:, None], -1).contiguous()
    if c["op"] == "moe_route_backward":
        st["dweights"] = torch.randn(T, k, device="cuda", generator=g)
        st["slope"] = 0.01 * torch.randn(E, device="cuda", generator=g)
        st["dloss"] = torch.rand((), device="cuda", generator=g) + 0.5
        st["dlogits"] = torch.empty_like(logits)
    return st


# ------------------------------------------------------------------ the framework's calls
def _run_own(st):
    import dense_gemm_tiled_amd as tg
    c = st["case"]
    if c["op"] == "cross_entropy":
        return tg.cross_entropy(st["x"], st["w"], st["targets"], scale=c["scale"])
    if c["op"] == "cross_entropy_backward":
        return tg.cross_entropy_backward(st["x"], st["w"], st["targets"], st["lse"], st["grad"], st["dx"],
                                         st["dw"], scale=c["scale"])
    if c["op"] == "moe_balance":
        return tg.moe_balance(st["logits"], st["ids"], coef=0.01)
    return tg.moe_route_backward(st["logits"], st["ids"], st["dweights"], st["dlogits"],
                                 renormalize=c["renorm"], scale=2.0, slope=st["slope"], dloss=st["dloss"])


# ------------------------------------------------------------------ plain forms
def _softmax(l, alive):
    """Softmax of the finite logits of the tokens that count, 0 elsewhere."""
    there = alive[:, None] & (l > -math.inf)
    l = torch.where(there, l, 0.0)
    m = torch.where(there, l, -math.inf).amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.where(there, torch.exp(l - m), 0.0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _plain(st):
    c = st["case"]
    if c["op"].startswith("cross"):
        x, w, targets = st["x"].float(), st["w"].float(), st["targets"]
        l = c["scale"] * (x @ w.t())
        counts = (targets >= 0) & (targets < c["V"])
        at = torch.where(counts, targets, 0)[:, None]
        if c["op"] == "cross_entropy":
            m = l.amax(1, keepdim=True)
            lse = (m + torch.log(torch.exp(l - m).sum(1, keepdim=True)))[:, 0]
            return torch.where(counts, lse - l.gather(1, at)[:, 0], 0.0), lse
        p = torch.exp(l - st["lse"][:, None])
        p = p - torch.zeros_like(p).scatter_(1, at, 1.0)
        p = c["scale"] * torch.where(counts, st["grad"], 0.0)[:, None] * p
        return (p @ w).to(st["x"].dtype), (p.t() @ x).to(st["w"].dtype)
    E, ids, l = c["E"], st["ids"], st["logits"].float()
    inside = (ids >= 0) & (ids < E)
    alive = inside.any(1)
    p = _softmax(l, alive)
    at = torch.where(inside, ids, E).long()
    if c["op"] == "moe_balance":
        counts = torch.zeros(E + 1, dtype=torch.int64, device=l.device)
        counts = counts.scatter_add_(0, at.flatten(), torch.ones_like(at).flatten())[:E]
        total, n = counts.sum(), alive.sum()
        share = counts.double() / total.clamp(min=1)
        loss = 0.01 * E * (share * p.double().sum(0)).sum() / n.clamp(min=1)
        slope = 0.01 * (E * counts - total).double() / (total * n).clamp(min=1)
        return loss.float(), counts.to(torch.int32), slope.float()
    chosen = torch.nn.functional.pad(p, (0, 1)).gather(1, at)            # p of each place, 0 for none
    if c["renorm"]:
        # from the logits themselves: the chosen ones' share of p may be small
        lc = torch.nn.functional.pad(torch.where(alive[:, None], l, -math.inf), (0, 1), value=-math.inf).gather(1, at)
        chosen = torch.exp(lc - lc.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
        chosen = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-30)
    wd = 2.0 * chosen * torch.where(inside, st["dweights"], 0.0)
    s = wd.sum(1, keepdim=True)
    d = torch.zeros(l.size(0), E + 1, device=l.device).scatter_add_(1, at, wd - chosen * s if c["renorm"] else wd)[:, :E]
    if not c["renorm"]:
        d = d - p * s
    d = d + st["dloss"] * p * (st["slope"] - (p * st["slope"]).sum(1, keepdim=True))
    return d.to(st["logits"].dtype)


def run(state):
    return _run_own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _exact_cross(st, c):
    """Token by token chunks, so that a large vocabulary fits."""
    w, s, V = st["w"].double(), c["scale"], c["V"]
    back = c["op"].endswith("backward")
    wt = w.t().contiguous()
    dw = torch.zeros_like(w) if back else None
    first, second = [], []
    for t0 in range(0, c["T"], 512):
        x, y = st["x"][t0:t0 + 512].double(), st["targets"][t0:t0 + 512]
        l = torch.matmul(x, wt) * s
        seen = (y >= 0) & (y < V)
        t = torch.nonzero(seen)[:, 0]
        if back:
            q = torch.exp(l - st["lse"][t0:t0 + 512].double()[:, None])
            q[t, y[t]] -= 1
            q *= (st["grad"][t0:t0 + 512].double() * seen * s)[:, None]
            first.append(torch.matmul(q, w))
            dw += torch.matmul(q.t().contiguous(), x)
        else:
            second.append(torch.logsumexp(l, 1))
            loss = torch.zeros(x.size(0), dtype=torch.float64, device=x.device)
            loss[t] = second[-1][t] - l[t, y[t]]
            first.append(loss)
    return torch.cat(first), dw if back else torch.cat(second)


def _exact_router(st, c):
    E, k, T = c["E"], c["k"], c["T"]
    ids, l = st["ids"].long(), st["logits"].double()
    named = torch.stack([(ids == e).sum(1) for e in range(E)], 1)        # [T, E] places of each expert
    alive = named.sum(1) > 0
    l = torch.where(torch.isfinite(l) & alive[:, None], l, -math.inf)
    z = torch.logsumexp(l, 1, keepdim=True)
    p = torch.where(z > -math.inf, torch.exp(l - torch.where(z > -math.inf, z, 0.0)), 0.0)
    if c["op"] == "moe_balance":
        counts, n = named.sum(0), int(alive.sum())
        total = int(counts.sum())
        if total == 0:
            zero = torch.zeros(E, dtype=torch.float64, device=l.device)
            return zero.sum(), counts.to(torch.int32), zero
        loss = 0.01 * E * torch.dot(counts.double() / total, p.mean(0) * (T / n))
        return loss, counts.to(torch.int32), 0.01 * (E * counts.double() / total - 1) / n
    out = st["dloss"].double() * (p * st["slope"].double() - p * (p @ st["slope"].double())[:, None])
    for j in range(k):
        # the j-th place's weight w_j = 2 q_j: dq_j = q_j (dl_j - sum_i q_i dl_i)
        t = torch.nonzero((ids[:, j] >= 0) & (ids[:, j] < E))[:, 0]
        e = ids[t, j]
        over = torch.where(named[t] > 0, l[t], -math.inf) if c["renorm"] else l[t]
        q = torch.exp(over - torch.logsumexp(over, 1, keepdim=True))
        mine = q[torch.arange(t.numel(), device=t.device), e][:, None]
        d = -q * mine
        d[torch.arange(t.numel(), device=t.device), e] += mine[:, 0]
        out[t] += 2.0 * st["dweights"][t, j].double()[:, None] * d
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_cross(st, case) if case["op"].startswith("cross") else _exact_router(st, case)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"].startswith("cross"):
        T, V, H, es = c["T"], c["V"], c["H"], _ES[c["dtype"]]
        once = (T + V) * H * es + T * 8
        if c["op"] == "cross_entropy":
            return {"bytes": once + T * 8, "flops": 2.0 * T * V * H}
        # the logits again, then two products; the gradients are as large as x and W
        return {"bytes": once + (T + V) * H * es + T * 8, "flops": 6.0 * T * V * H}
    T, E, k, es = c["T"], c["E"], c["k"], _ES[c["dtype"]]
    if c["op"] == "moe_balance":
        return {"bytes": T * (E * es + k * 4) + E * 8, "flops": 4.0 * T * E}
    return {"bytes": T * (2 * E * es + k * 8) + E * 4, "flops": 8.0 * T * E}
