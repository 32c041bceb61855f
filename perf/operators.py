"""Cases and plain forms of the training-step operators: the AdamW step over
many tensors at once (states in 32 or in 8 bits, with the gradient norm that
clips it) and the expert router (top-k choice, gate weights, per-expert counts
and the balance loss, with their gradients).

`run(state)` computes an operator by elementary torch operations, or, where
`own` is true, by this repository's package, on what `prepare` made.

AdamW, per element, t the number of this step (decoupled weight decay):

    norm = sqrt(sum g^2) over every tensor;  c = min(1, max_norm / norm)
    m' = b1 m + (1 - b1) c g        v' = b2 v + (1 - b2) (c g)^2
    p' = p - lr (wd p + (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps))

States in 8 bits are kept in blocks of 256 elements of a tensor, one float32
scale a block, with square-law codes: m = a q |q|, q in [-127, 127], where
a = max |m'| / 127^2; v = (r u^2)^2, u in [0, 255], where r = sqrt(max v') /
255^2.  Each value is held as the code nearest to it (nearest in m and in
sqrt(v); a tie goes to the smaller code; a positive v never to 0).  p' is taken
from m' and v' before they are coded.

Router, per token with logits x over E experts, K of them chosen:

    p = softmax(x);  chosen: the K largest finite x (ties to the lowest index)
    w = p of the chosen ones (divided by their sum where `renormalize` is true)
    C_e = tokens that chose e (per rank);  S_e = sum of p_e;  T = tokens
    loss = E / (K T^2) sum_e C_e S_e        (C, S, T over all ranks' tokens)

A masked token is no token: index -1, weight 0, gradient 0.  The gradient is
that of sum(dw * w) + dloss * loss with respect to x, C held fixed.
"""

import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}

BLOCK = 256                       # elements under one scale
LR, B1, B2, EPS, WD, MAX_NORM = 1e-3, 0.9, 0.999, 1e-8, 0.1, 1.0
STEPS_BEFORE = 100                # steps taken before the one that is measured


def listed():
    return [
        # one normalisation vector: what a call costs when it moves nothing
        {"name": "adamw vector", "op": "adamw", "tensors": 1, "elements": 1000,
         "param": "float32", "grad": "float32", "copy": False},
        # the tensors of a small model, matrices and vectors of odd sizes,
        # bfloat16 gradients and bfloat16 working copies
        {"name": "adamw many tensors", "op": "adamw", "tensors": 250, "elements": 9_000_001,
         "param": "float32", "grad": "bfloat16", "copy": True},
        # eight ranks' shards of a 1.2 GB float32 gradient after its ReduceScatter
        {"name": "adamw shards", "op": "adamw", "tensors": 8, "elements": 300_000_000,
         "param": "float32", "grad": "float32", "copy": True},
        # one small tensor whose last block is short
        {"name": "adamw8 small", "op": "adamw8", "tensors": 1, "elements": 10_007,
         "param": "float32", "grad": "float32", "copy": False},
        # a 25 MB gradient bucket
        {"name": "adamw8 bucket", "op": "adamw8", "tensors": 12, "elements": 6_553_600,
         "param": "float32", "grad": "float32", "copy": False},
        # eight shards again, states in 8 bits, bfloat16 gradients and copies
        {"name": "adamw8 shards", "op": "adamw8", "tensors": 8, "elements": 300_000_000,
         "param": "float32", "grad": "bfloat16", "copy": True},
        # one token being decoded
        {"name": "route one token", "op": "route", "ranks": 1, "tokens": 1, "experts": 8,
         "top_k": 2, "dtype": "bfloat16", "renormalize": True, "masked": 0.0},
        # a batch of prompts spread over eight ranks
        {"name": "route batch", "op": "route", "ranks": 8, "tokens": 509, "experts": 64,
         "top_k": 6, "dtype": "float32", "renormalize": False, "masked": 0.1},
        # a long prefill: every rank a full sequence, many small experts
        {"name": "route long", "op": "route", "ranks": 8, "tokens": 16_384, "experts": 256,
         "top_k": 8, "dtype": "bfloat16", "renormalize": True, "masked": 0.0},
        # a small training batch with an odd number of experts
        {"name": "route train small", "op": "route_train", "ranks": 2, "tokens": 100,
         "experts": 61, "top_k": 4, "dtype": "float32", "renormalize": False, "masked": 0.2},
        # the ordinary training micro-batch: 4,096 tokens a rank, two experts each
        {"name": "route train", "op": "route_train", "ranks": 8, "tokens": 4096, "experts": 128,
         "top_k": 2, "dtype": "bfloat16", "renormalize": True, "masked": 0.05},
        # the largest: long sequences, 256 experts, float32 logits
        {"name": "route train long", "op": "route_train", "ranks": 8, "tokens": 16_384,
         "experts": 256, "top_k": 8, "dtype": "float32", "renormalize": False, "masked": 0.05},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adamw", "adamw8", "route", "route_train"])
    if op.startswith("adamw"):
        elements = _log_uniform(rng, 1000, 250_000_000)
        param = rng.choice(["float32", "float32", "bfloat16"])
        return {"op": op, "tensors": _log_uniform(rng, 1, min(400, elements // 100)),
                "elements": elements, "param": param,
                "grad": rng.choice(["float32", "bfloat16"]),
                "copy": param == "float32" and rng.random() < 0.5}
    ranks = _log_uniform(rng, 1, 16)
    experts = _log_uniform(rng, 4, 512)
    tokens = _log_uniform(rng, 1, min(16_384, 2 ** 25 // (ranks * experts)))
    return {"op": op, "ranks": ranks, "tokens": tokens, "experts": experts,
            "top_k": rng.randint(1, min(8, experts)),
            "dtype": rng.choice(["float32", "bfloat16"]), "renormalize": rng.random() < 0.5,
            "masked": rng.choice([0.0, 0.05, 0.5])}


def _sizes(case):
    """Sizes of the tensors: uneven, at least one element each, `elements` in all."""
    n, total = case["tensors"], case["elements"]
    rng = random.Random(n * 1_000_003 + total)
    cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _spans(case):
    """(begin, end) of each tensor in flat buffers where each begins on a block; their length."""
    sizes = _sizes(case)
    room = [-(-s // BLOCK) * BLOCK for s in sizes]
    starts = [sum(room[:i]) for i in range(len(room))]
    return [(b, b + s) for b, s in zip(starts, sizes)], sum(room)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    if case["op"] in ("adamw", "adamw8"):
        return _prepare_adamw(case, gen)
    shape = (case["ranks"], case["tokens"], case["experts"])
    bias = torch.randn(shape[2], generator=gen, device=DEVICE) * 0.5      # some experts draw more
    x = torch.randn(shape, generator=gen, device=DEVICE) * 1.5 + bias
    # one row in fifty has experts ruled out, now and then all of them
    out = torch.rand(shape[:2], generator=gen, device=DEVICE) < 0.02
    share = torch.rand(shape[:2], generator=gen, device=DEVICE) * 1.2
    x = torch.where(out[..., None] & (torch.rand(shape, generator=gen, device=DEVICE) < share[..., None]),
                    -math.inf, x).to(DTYPES[case["dtype"]])
    state = {"case": case, "logits": x, "ranks": list(x), "mask": None, "masks": None}
    if case["masked"]:
        state["mask"] = torch.rand(shape[:2], generator=gen, device=DEVICE) >= case["masked"]
        state["masks"] = list(state["mask"])
    if case["op"] == "route_train":
        state["dweights"] = torch.randn(shape[:2] + (case["top_k"],), generator=gen, device=DEVICE) * 1e-3
        state["dweights_ranks"] = list(state["dweights"])
        state["dloss"] = torch.full((), 0.01, device=DEVICE)
    return state


def _prepare_adamw(case, gen):
    spans, room = _spans(case)
    live = torch.zeros(room, dtype=torch.bool, device=DEVICE)
    [live[a:b].fill_(True) for a, b in spans]

    def normal(std):
        return torch.where(live, torch.randn(room, generator=gen, device=DEVICE) * std, 0.0)

    p = normal(0.02).to(DTYPES[case["param"]])
    g = normal(1e-3).to(DTYPES[case["grad"]])
    m = normal(3e-4)
    v = torch.where(live, torch.rand(room, generator=gen, device=DEVICE).square() * 2e-6, 0.0)
    state = {"case": case, "p": p, "g": g, "steps": STEPS_BEFORE,
             "copy": torch.zeros(room, dtype=torch.bfloat16, device=DEVICE) if case["copy"] else None}
    if case["op"] == "adamw":
        state |= {"m": m, "v": v}
    else:
        state["m"], state["a"] = _code_m(m.double().view(-1, BLOCK))
        state["v"], state["r"] = _code_v(v.double().view(-1, BLOCK))
    if own:
        import tree_allreduce_algorithms_amd as ar
        cut = lambda t: [t[a:b] for a, b in spans]  # noqa: E731
        cut_scale = lambda t: [t[a // BLOCK:-(-b // BLOCK)] for a, b in spans]  # noqa: E731
        held = {"exp_avg": cut(state["m"]), "exp_avg_sq": cut(state["v"])}
        if case["op"] == "adamw8":
            held |= {"exp_avg_scale": cut_scale(state["a"]), "exp_avg_sq_scale": cut_scale(state["r"])}
        state["optimizer"] = ar.AdamW(
            cut(p), cut(g), copies=cut(state["copy"]) if case["copy"] else None,
            state_bits=8 if case["op"] == "adamw8" else 32, state=held, steps=STEPS_BEFORE,
            betas=(B1, B2), eps=EPS, weight_decay=WD)
    return state


# --- plain forms -----------------------------------------------------------------

def _code_m(m):
    """Signed square-law codes of the rows of m (float64), and the rows' scales."""
    a = (m.abs().amax(-1, keepdim=True) / 127 ** 2).float()
    t = torch.where(a > 0, m.abs() / torch.where(a > 0, a, 1.0).double(), 0.0)
    q = t.sqrt().floor()
    q = torch.where(t > q * q + q + 0.5, q + 1, q).clamp(max=127)
    return torch.where(m < 0, -q, q).to(torch.int8).view(-1), a.view(-1)


def _code_v(v):
    """Square-law codes of the square roots of the rows of v (float64), and the rows' scales."""
    s = v.sqrt()
    r = (s.amax(-1, keepdim=True) / 255 ** 2).float()
    t = torch.where(r > 0, s / torch.where(r > 0, r, 1.0).double(), 0.0)
    u = t.sqrt().floor()
    u = torch.where(t > u * u + u + 0.5, u + 1, u).clamp(max=255)
    return torch.where((t > 0) & (u == 0), 1.0, u).to(torch.uint8).view(-1), r.view(-1)


def _values_m(q, a):
    q = q.view(-1, BLOCK).double()
    return q * q.abs() * a.double()[:, None]


def _values_v(u, r):
    u = u.view(-1, BLOCK).double()
    return (u * u * r.double()[:, None]).square()


def _plain_adamw(s):
    s["steps"] += 1
    norm = s["g"].double().square().sum().sqrt()
    c = torch.where(norm > MAX_NORM, MAX_NORM / norm, 1.0).float()
    bc1, bc2 = 1 - B1 ** s["steps"], 1 - B2 ** s["steps"]
    if s["case"]["op"] == "adamw":
        g = s["g"].float() * c
        m = s["m"].copy_(B1 * s["m"] + (1 - B1) * g)
        v = s["v"].copy_(B2 * s["v"] + (1 - B2) * g * g)
        held = {"m": m, "v": v}
    else:
        # 64 bits: a code changes where a value crosses the middle between two
        g = s["g"].double().view(-1, BLOCK) * c.double()
        m = B1 * _values_m(s["m"], s["a"]) + (1 - B1) * g
        v = B2 * _values_v(s["v"], s["r"]) + (1 - B2) * g * g
        for_m, for_v = _code_m(m), _code_v(v)
        s["m"].copy_(for_m[0]), s["a"].copy_(for_m[1]), s["v"].copy_(for_v[0]), s["r"].copy_(for_v[1])
        held = {"m": _values_m(s["m"], s["a"]).float().view(-1),
                "v": _values_v(s["v"], s["r"]).float().view(-1)}
        m, v = m.float().view(-1), v.float().view(-1)
    p = s["p"].float()
    p = p - LR * (WD * p + (m / bc1) / ((v / bc2).sqrt() + EPS))
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    return {"norm": norm.float(), "p": s["p"], "copy": s["copy"], **held}


def _plain_route(s):
    case = s["case"]
    k, experts = case["top_k"], case["experts"]
    x = s["logits"].float()
    if s["mask"] is not None:
        x = torch.where(s["mask"][..., None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    live = top > -math.inf
    e = (x - torch.where(live, top, 0.0)).exp()
    p = e / torch.where(live, e.sum(-1, keepdim=True), 1.0)
    value, index = x.sort(dim=-1, descending=True, stable=True)      # ties: the lowest index first
    value, index = value[..., :k], index[..., :k]
    chosen = value > -math.inf
    w = torch.where(chosen, p.gather(-1, index), 0.0)
    if case["renormalize"]:
        w = w / torch.where(live, w.sum(-1, keepdim=True), 1.0)
    counts = torch.zeros((case["ranks"], experts), dtype=torch.int32, device=x.device)
    counts.scatter_add_(1, index.flatten(1), chosen.flatten(1).int())
    tokens = live.sum()
    share = experts * counts.sum(0).double() / (k * tokens.clamp(min=1).double() ** 2)
    loss = (share * p.sum((0, 1), dtype=torch.float64)).sum().float()
    out = {"indices": torch.where(chosen, index, -1).int(), "weights": w, "counts": counts, "loss": loss}
    if case["op"] == "route_train":
        coef = (s["dloss"].double() * share).float()
        at = lambda d: torch.zeros_like(p).scatter_(-1, index, torch.where(chosen, d, 0.0))  # noqa: E731
        dw = s["dweights"]
        if case["renormalize"]:
            dx = p * (coef - (p * coef).sum(-1, keepdim=True)) + at(w * (dw - (w * dw).sum(-1, keepdim=True)))
        else:
            dp = coef + at(dw)
            dx = p * (dp - (p * dp).sum(-1, keepdim=True))
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


# --- the framework's calls ---------------------------------------------------------

def _own_adamw(s):
    import tree_allreduce_algorithms_amd as ar
    opt = s["optimizer"]
    norm = opt.grad_norm(max_norm=MAX_NORM)
    opt.step(lr=LR, clip=True)
    if s["case"]["op"] == "adamw":
        held = {"m": s["m"], "v": s["v"]}
    else:
        held = {"m": ar.dequantize(s["m"], s["a"]), "v": ar.dequantize(s["v"], s["r"])}
    return {"norm": norm, "p": s["p"], "copy": s["copy"], **held}


def _own_route(s):
    import tree_allreduce_algorithms_amd as ar
    case = s["case"]
    r = ar.route(s["ranks"], case["top_k"], mask=s["masks"], renormalize=case["renormalize"])
    out = {"indices": r.indices, "weights": r.weights, "counts": r.counts, "loss": r.loss}
    if case["op"] == "route_train":
        out["dlogits"] = ar.route_grad(s["ranks"], r, dweights=s["dweights_ranks"], dloss=s["dloss"])
    return out


def run(state):
    if state["case"]["op"] in ("adamw", "adamw8"):
        return _own_adamw(state) if own else _plain_adamw(state)
    return _own_route(state) if own else _plain_route(state)


# --- what a pass cannot do without ---------------------------------------------------

def work(case):
    size = {"float32": 4, "bfloat16": 2}
    if case["op"] in ("adamw", "adamw8"):
        n, blocks = case["elements"], sum(-(-s // BLOCK) for s in _sizes(case))
        each = 2 * size[case["param"]] + size[case["grad"]] + (2 if case["copy"] else 0)
        # states in 32 bits: read and written; in 8: read and written, and given as values
        held = 16 * n if case["op"] == "adamw" else (4 + 8) * n + 16 * blocks
        return {"bytes": each * n + held, "flops": (20 if case["op"] == "adamw" else 45) * n}
    tokens = case["ranks"] * case["tokens"]
    n, s = tokens * case["experts"], size[case["dtype"]]
    nbytes = n * s + tokens * case["top_k"] * 8 + (tokens if case["masked"] else 0) \
        + case["ranks"] * case["experts"] * 4
    flops = n * (4 + case["top_k"])
    if case["op"] == "route_train":
        nbytes += n * s + tokens * case["top_k"] * 4
        flops += n * 6
    return {"bytes": nbytes, "flops": flops}


# --- the definitions, in 64 bits -------------------------------------------------------

def _nearest(t, codes):
    """Index of the entry of `codes` (ascending) nearest to each t, the lower one at a tie."""
    return torch.bucketize(t, (codes[1:] + codes[:-1]) / 2)


def _exact_adamw(case, s):
    f64 = torch.float64
    g = s["g"].to(f64)
    norm = torch.linalg.vector_norm(g)
    # the factor is a float32 number, which the norm and its bound give
    c = float(torch.tensor(min(1.0, MAX_NORM / max(float(norm), 1e-300)), dtype=torch.float32))
    g = g * c
    if case["op"] == "adamw":
        m, v = s["m"].to(f64), s["v"].to(f64)
    else:
        m = s["m"].to(f64)
        m = torch.sign(m) * m ** 2 * s["a"].to(f64).repeat_interleave(BLOCK)
        v = s["v"].to(f64) ** 4 * s["r"].to(f64).repeat_interleave(BLOCK) ** 2
    m.mul_(B1).add_(g, alpha=1 - B1)
    v.mul_(B2).addcmul_(g, g, value=1 - B2)
    t = STEPS_BEFORE + 1
    step = (m / (1 - B1 ** t)).div_((v / (1 - B2 ** t)).sqrt_().add_(EPS))
    p = s["p"].to(f64)
    p = p * (1 - LR * WD) - LR * step
    del step, g
    if case["op"] == "adamw8":
        squares = torch.arange(256, dtype=f64, device=DEVICE) ** 2
        a = (m.view(-1, BLOCK).abs().amax(1) / squares[127]).float().to(f64).repeat_interleave(BLOCK)
        m = torch.sign(m) * a * squares[_nearest(torch.nan_to_num(m.abs() / a), squares[:128])]
        v = v.sqrt_()
        r = (v.view(-1, BLOCK).amax(1) / squares[255]).float().to(f64).repeat_interleave(BLOCK)
        code = _nearest(torch.nan_to_num(v / r), squares)
        code = torch.where(v > 0, code.clamp_(min=1), 0)
        v = (r * squares[code]).square()
    return {"norm": norm, "p": p, "copy": p if case["copy"] else None, "m": m, "v": v}


def _exact_route(case, s):
    k, experts = case["top_k"], case["experts"]
    x = s["logits"].to(torch.float64).reshape(-1, experts)
    alive = torch.isfinite(x).any(1)
    if s["mask"] is not None:
        alive &= s["mask"].reshape(-1)
    x = x[alive].requires_grad_(case["op"] == "route_train")
    p = torch.softmax(x, 1)
    left, picks = x.detach().clone(), []
    for _ in range(k):
        best = left.argmax(1, keepdim=True)                       # the first of equal ones
        picks.append(torch.where(left.gather(1, best) > -math.inf, best, -1))
        left.scatter_(1, best, -math.inf)
    pick = torch.cat(picks, 1)
    chosen = pick >= 0
    w = p.gather(1, pick.clamp(min=0)) * chosen
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    rows = case["ranks"] * case["tokens"]
    index = torch.full((rows, k), -1, dtype=torch.int32, device=x.device)
    index[alive] = pick.int()
    rank = torch.arange(case["ranks"], device=x.device).repeat_interleave(case["tokens"])[alive]
    slot = (rank[:, None] * experts + pick)[chosen]
    counts = torch.bincount(slot, minlength=case["ranks"] * experts).reshape(case["ranks"], experts)
    tokens = max(1, int(alive.sum()))
    # the loss from the shares of the load and of the probabilities, E f . P
    loss = experts * (counts.sum(0) / (k * tokens) * (p.sum(0) / tokens)).sum()
    weights = torch.zeros((rows, k), dtype=torch.float64, device=x.device)
    weights[alive] = w.detach()
    shape = (case["ranks"], case["tokens"])
    out = {"indices": index.view(*shape, k), "weights": weights.view(*shape, k),
           "counts": counts.int(), "loss": loss.detach()}
    if case["op"] == "route_train":
        dx = torch.zeros((rows, experts), dtype=torch.float64, device=x.device)
        if bool(alive.any()):
            dw = s["dweights"].to(torch.float64).reshape(rows, k)[alive]
            ((w * dw).sum() + float(s["dloss"]) * loss).backward()
            dx[alive] = x.grad
        out["dlogits"] = dx.view(*shape, experts)
    return out


def exact(case, seed):
    """What run() gives for these inputs, from the definitions in 64 bits."""
    s = prepare(case, seed)
    return _exact_adamw(case, s) if case["op"] in ("adamw", "adamw8") else _exact_route(case, s)
