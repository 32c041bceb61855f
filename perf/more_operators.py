"""Cases and plain forms of the operators that follow the expert router and
stand beside AdamW: the products of the chosen experts (the order of the pairs
by expert, the products grouped by expert, the weighted sum back to the tokens,
and all their gradients) and the Muon step (momentum, its orthogonalisation by
Newton-Schulz products, the update).

`run(state)` computes an operator by elementary torch operations, or, where
`own` is true, by this repository's package, on what `prepare` made.

Experts.  A pair p = t K + k is the k-th choice of token t, of expert e(p) (or
none, -1).  Rows are the pairs in order: by expert, within an expert by p, those
without one at the end.  With x [tokens, in], W [experts, in, out], weights w:

    y_i = x_t(i) W_e(i)                   rows without an expert are 0
    out_t = sum_k w_tk y_row(t,k)         over the pairs that have an expert

    dy_i = w_p(i) dout_t(i)               dw_tk = dout_t . y_row(t,k)
    dx_t = sum_k dy_row(t,k) W_e(t,k)^T   dW_e = sum over e's rows of x_t(i)^T dy_i

Each of y, out, dy, the rows of dy W^T, and dx is a tensor of the inputs' type,
so each is rounded to it once; dw and dW are float32.

Muon, per matrix (the last two dimensions), with s = sqrt(max(1, rows / cols)):

    m' = mu m + g;  u = g + mu m';  X = u / (|u| + 1e-7)
    five times: A = X X^T, X = a X + (b A + c A A) X
    p' = p - lr (wd p + s X)              X X^T by the shorter side of u
"""

import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}

LR, MU, WD, STEPS, EPS = 0.02, 0.95, 0.1, 5, 1e-7
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # one token being decoded: two experts' weights are read, latency counts
        {"name": "experts one token", "op": "experts", "tokens": 1, "experts": 8, "top_k": 2,
         "in": 1024, "out": 1024, "masked": 0.0},
        # 32 requests being decoded over many small experts
        {"name": "experts decode", "op": "experts", "tokens": 32, "experts": 64, "top_k": 6,
         "in": 2048, "out": 1024, "masked": 0.0},
        # a padded batch of prompts, an odd number of experts, odd sizes
        {"name": "experts odd batch", "op": "experts", "tokens": 509, "experts": 61, "top_k": 4,
         "in": 1001, "out": 777, "masked": 0.1},
        # a long prefill
        {"name": "experts prefill", "op": "experts", "tokens": 16_384, "experts": 128, "top_k": 8,
         "in": 2048, "out": 1024, "masked": 0.0},
        # the backward pass of a small training batch
        {"name": "experts train small", "op": "experts_grad", "tokens": 200, "experts": 8, "top_k": 2,
         "in": 256, "out": 512, "masked": 0.2},
        # odd sizes again, in training
        {"name": "experts train odd", "op": "experts_grad", "tokens": 1021, "experts": 61, "top_k": 4,
         "in": 515, "out": 1030, "masked": 0.05},
        # the ordinary training micro-batch, two of 64 experts a token
        {"name": "experts train", "op": "experts_grad", "tokens": 4096, "experts": 64, "top_k": 2,
         "in": 1024, "out": 2048, "masked": 0.05},
        # the largest: long sequences, eight of 128 experts a token
        {"name": "experts train long", "op": "experts_grad", "tokens": 16_384, "experts": 128, "top_k": 8,
         "in": 2048, "out": 1024, "masked": 0.0},
        # one small matrix of odd sizes: what a step costs when it computes little
        {"name": "muon small", "op": "muon", "shapes": "1x100x61", "param": "float32",
         "grad": "float32", "copy": False},
        # the matrices of a small layer, bfloat16 gradients and working copies
        {"name": "muon layer", "op": "muon", "shapes": "4x1024x1024,1x4096x1024,1x1024x4096",
         "param": "float32", "grad": "bfloat16", "copy": True},
        # the weights of many experts, sums of gradients in float32
        {"name": "muon experts", "op": "muon", "shapes": "64x1024x512", "param": "float32",
         "grad": "float32", "copy": True},
        # the largest: matrices of a wide model
        {"name": "muon large", "op": "muon", "shapes": "2x4096x4096,1x8192x4096", "param": "bfloat16",
         "grad": "bfloat16", "copy": False},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size of the range: as it comes, or (three times of five) a multiple of 64 where it is long enough."""
    n = _log_uniform(rng, lo, hi)
    return n // 64 * 64 if n >= 64 and rng.random() < 0.6 else n


def draw(rng):
    if rng.random() < 0.4:
        param = rng.choice(["float32", "float32", "bfloat16"])
        shapes, left = [], 2e11              # products m^2 n + m^3 + 2 m^2 n of a Newton-Schulz step
        for _ in range(rng.randint(1, 4)):
            r, c = _size(rng, 16, 4096), _size(rng, 16, 4096)
            m, n = min(r, c), max(r, c)
            most = min(64, int(left / (3 * m * m * n + m ** 3)))
            if most < 1:
                continue
            count = _log_uniform(rng, 1, most)
            left -= count * (3 * m * m * n + m ** 3)
            shapes.append(f"{count}x{r}x{c}")
        return {"op": "muon", "shapes": ",".join(shapes) or "1x1024x1000", "param": param,
                "grad": rng.choice(["float32", "bfloat16"]),
                "copy": param == "float32" and rng.random() < 0.5}
    experts = _log_uniform(rng, 4, 256)
    k = rng.randint(1, min(8, experts))
    rows = _size(rng, 32, 2048)
    cols = _size(rng, 32, min(2048, 2 ** 28 // (experts * rows)))
    most = min(16_384, 2 ** 38 // (k * rows * cols))
    return {"op": rng.choice(["experts", "experts_grad"]), "tokens": _log_uniform(rng, 1, most),
            "experts": experts, "top_k": k, "in": rows, "out": cols,
            "masked": rng.choice([0.0, 0.05, 0.5])}


def _shapes(case):
    """(count, rows, cols) of each tensor of a Muon case."""
    return [tuple(int(n) for n in s.split("x")) for s in case["shapes"].split(",")]


def _views(case, flat):
    """The tensors of a Muon case in a flat buffer."""
    shapes = _shapes(case)
    return [t.view(s) for t, s in zip(flat.split([math.prod(s) for s in shapes]), shapes)]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=DEVICE) * std

    if case["op"] == "muon":
        return _prepare_muon(case, normal)
    t, e, k, i, o = (case[n] for n in ("tokens", "experts", "top_k", "in", "out"))
    logits = normal(t, e, std=1.5) + normal(e, std=0.5)                  # some experts draw more
    value, index = logits.topk(k, dim=-1)
    none = torch.rand(t, 1, generator=gen, device=DEVICE) < case["masked"]
    state = {"case": case, "indices": torch.where(none, -1, index).int(),
             "weights": torch.where(none, 0.0, value.softmax(-1)),
             "x": normal(t, i).bfloat16(), "w": normal(e, i, o, std=i ** -0.5).bfloat16()}
    if case["op"] == "experts_grad":
        # the forward pass's rows and the gradient of its sums
        state["y"] = torch.where(_order(state["indices"], e)[1][-1] > torch.arange(t * k, device=DEVICE)[:, None],
                                 normal(t * k, o), 0.0).bfloat16()
        state["dout"] = normal(t, o, std=1e-3).bfloat16()
    return state


def _prepare_muon(case, normal):
    parts = []
    for n, r, c in _shapes(case):
        # a gradient: few strong directions and noise
        rank = max(1, min(r, c) // 16)
        strong = torch.matmul(normal(n, r, rank) * torch.arange(1, rank + 1, device=DEVICE).float() ** -0.5,
                              normal(n, rank, c))
        parts.append((strong * rank ** -0.5 + normal(n, r, c, std=0.2)).flatten() * 1e-3)
    g = torch.cat(parts).to(DTYPES[case["grad"]])
    state = {"case": case, "g": g, "p": normal(g.numel(), std=0.02).to(DTYPES[case["param"]]),
             "m": torch.cat([(p * 8 + normal(p.numel(), std=1e-3)) for p in parts]),
             "copy": torch.zeros(g.numel(), dtype=torch.bfloat16, device=DEVICE) if case["copy"] else None}
    if own:
        import tree_allreduce_algorithms_amd as ar
        state["optimizer"] = ar.Muon(
            _views(case, state["p"]), _views(case, g),
            copies=_views(case, state["copy"]) if case["copy"] else None,
            state={"momentum": _views(case, state["m"])}, momentum=MU, nesterov=True, ns_steps=STEPS,
            eps=EPS, weight_decay=WD)
    return state


# --- plain forms -----------------------------------------------------------------

def _order(indices, experts):
    """The pairs in order (-1 behind the last that has an expert), and where each expert's begin."""
    e = indices.flatten().long()
    key = torch.where(e >= 0, e, experts)
    order = key.argsort(stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=e.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:experts].cumsum(0)])
    return order, offsets


def _grouped(offsets, rows):
    """A padded place [expert, slot] for every row that has an expert, and the slots."""
    live = int(offsets[-1])
    counts = offsets[1:] - offsets[:-1]
    expert = torch.repeat_interleave(torch.arange(counts.numel(), device=offsets.device), counts, output_size=live)
    return live, expert, torch.arange(live, device=offsets.device) - offsets[expert], int(counts.max()) if rows else 0


def _products(x, w, place):
    """x's rows times their expert's matrix, in float32 (a padded batch); 0 behind the last."""
    live, expert, slot, room = place
    out = torch.zeros((x.shape[0], w.shape[2]), device=x.device)
    if live:
        padded = torch.zeros((w.shape[0], room, w.shape[1]), device=x.device)
        padded[expert, slot] = x[:live].float()
        out[:live] = torch.bmm(padded, w.float())[expert, slot]
    return out


def _plain_experts(s):
    case, k = s["case"], s["case"]["top_k"]
    order, offsets = _order(s["indices"], case["experts"])
    place = _grouped(offsets, order.numel())
    live, dtype = place[0], s["x"].dtype
    token = order // k
    row = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device)).view(-1, k)
    chosen = (row < live)[..., None]
    gather = lambda rows: torch.where(chosen, rows.float()[row], 0.0)  # noqa: E731  [tokens, top_k, size]
    if case["op"] == "experts":
        y = _products(s["x"][token], s["w"], place).to(dtype)
        out = (s["weights"][..., None] * gather(y)).sum(1).to(dtype)
        pairs = torch.where(torch.arange(order.numel(), device=order.device) < live, order, -1).int()
        return {"order": pairs, "offsets": offsets.int(), "y": y, "out": out}
    dout = s["dout"].float()
    dy = s["weights"].flatten()[order][:, None] * dout[token]
    dy[live:] = 0.0
    dy = dy.to(dtype)
    dweights = (dout[:, None] * gather(s["y"])).sum(-1)
    dx = gather(_products(dy, s["w"].transpose(1, 2), place).to(dtype)).sum(1).to(dtype)
    dw = torch.zeros(s["w"].shape, device=dout.device)
    if live:
        expert, slot, room = place[1:]
        xs, ds = (torch.zeros((case["experts"], room, n), device=dout.device) for n in (case["in"], case["out"]))
        xs[expert, slot], ds[expert, slot] = s["x"][token[:live]].float(), dy[:live].float()
        dw = torch.bmm(xs.transpose(1, 2), ds)
    return {"dy": dy, "dweights": dweights, "dx": dx, "dw": dw}


def _plain_muon(s):
    case, (a, b, c) = s["case"], COEFFICIENTS
    g = s["g"].float()
    s["m"].mul_(MU).add_(g)
    for p, copy, u in zip(_views(case, s["p"]), _views(case, s["copy"]) if case["copy"] else _shapes(case),
                          _views(case, g + MU * s["m"])):
        x = u / (u.double().square().sum((1, 2), keepdim=True).sqrt() + EPS).float()
        tall = x.shape[1] > x.shape[2]
        x = x.transpose(1, 2).contiguous() if tall else x
        for _ in range(STEPS):
            gram = torch.bmm(x, x.transpose(1, 2))
            x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
        x = x.transpose(1, 2) if tall else x
        scale = max(1.0, x.shape[1] / x.shape[2]) ** 0.5
        new = p.float() - LR * (WD * p.float() + scale * x)
        p.copy_(new)
        if case["copy"]:
            copy.copy_(new)
    return {"p": s["p"], "copy": s["copy"], "m": s["m"]}


# --- the framework's calls ---------------------------------------------------------

def _own_experts(s):
    import tree_allreduce_algorithms_amd as ar
    o = ar.expert_order(s["indices"], s["case"]["experts"])
    if s["case"]["op"] == "experts":
        y = ar.expert_matmul(s["x"], s["w"], o, gather=True)
        return {"order": o.order, "offsets": o.offsets, "y": y, "out": ar.expert_combine(y, o, s["weights"])}
    dy, dweights = ar.expert_combine_grad(s["dout"], s["y"], o, s["weights"])
    dx = ar.expert_combine(ar.expert_matmul(dy, s["w"].transpose(1, 2), o), o)
    return {"dy": dy, "dweights": dweights, "dx": dx, "dw": ar.expert_weight_grad(s["x"], dy, o, gather=True)}


def _own_muon(s):
    s["optimizer"].step(lr=LR)
    return {"p": s["p"], "copy": s["copy"], "m": s["m"]}


def run(state):
    if state["case"]["op"] == "muon":
        return _own_muon(state) if own else _plain_muon(state)
    return _own_experts(state) if own else _plain_experts(state)


# --- what a pass cannot do without ---------------------------------------------------

def work(case):
    size = {"float32": 4, "bfloat16": 2}
    if case["op"] == "muon":
        flops = nbytes = 0
        for n, r, c in _shapes(case):
            short, long = min(r, c), max(r, c)
            # A and A A are symmetric: half of each; and X by the sum
            flops += n * STEPS * (short * short * long + short ** 3 + 2 * short * short * long)
            nbytes += n * r * c * (2 * size[case["param"]] + size[case["grad"]] + 8 + (2 if case["copy"] else 0))
        return {"bytes": nbytes, "flops": flops}
    t, e, k, i, o = (case[n] for n in ("tokens", "experts", "top_k", "in", "out"))
    pairs = int(t * k * (1 - case["masked"])) or 1
    used = min(e, pairs)                      # at most so many experts' weights are needed
    if case["op"] == "experts":
        return {"bytes": 2 * (t * i + used * i * o + t * k * o + t * o) + t * k * 12, "flops": 2 * pairs * i * o}
    return {"bytes": 2 * (t * o + 2 * t * k * o + used * i * o + 2 * t * i) + 4 * e * i * o + t * k * 12,
            "flops": 4 * pairs * i * o + 3 * pairs * o}


# --- the definitions, in 64 bits -------------------------------------------------------

def _exact_experts(case, s):
    k, e = case["top_k"], case["experts"]
    pair_expert = s["indices"].reshape(-1)
    lists = [torch.nonzero(pair_expert == j).flatten() for j in range(e)]
    order = torch.cat(lists)
    live = order.numel()
    ends = torch.tensor([0] + [p.numel() for p in lists]).cumsum(0).tolist()
    x, w, gate = s["x"].double(), s["w"], s["weights"].double().reshape(-1)
    rows = pair_expert.numel()
    if case["op"] == "experts":
        y = torch.zeros((rows, case["out"]), dtype=torch.float64, device=x.device)
        out = torch.zeros((case["tokens"], case["out"]), dtype=torch.float64, device=x.device)
        for j, p in enumerate(lists):
            if p.numel():
                y[ends[j]:ends[j + 1]] = x[p // k] @ w[j].double()
                out.index_add_(0, p // k, gate[p, None] * y[ends[j]:ends[j + 1]])
        order = torch.cat([order, order.new_full((rows - live,), -1)]).int()
        return {"order": order, "offsets": torch.tensor(ends, dtype=torch.int32, device=x.device), "y": y, "out": out}
    dout, y = s["dout"].double(), s["y"]
    dy = torch.zeros((rows, case["out"]), dtype=torch.float64, device=x.device)
    dgate = torch.zeros(rows, dtype=torch.float64, device=x.device)
    dx, dw = torch.zeros_like(x), torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    for j, p in enumerate(lists):
        if p.numel():
            at = slice(ends[j], ends[j + 1])
            up = dout[p // k]
            dy[at] = gate[p, None] * up
            dgate[p] = torch.linalg.vecdot(up, y[at].double())
            # the gradients' products take dy as the tensor that it is, a float32 product in bfloat16
            held = dy[at].float().bfloat16().double()
            dx.index_add_(0, p // k, held @ w[j].double().t())
            dw[j] = x[p // k].t() @ held
    return {"dy": dy, "dweights": dgate.view(-1, k), "dx": dx, "dw": dw}


def _exact_muon(case, s):
    # the same polynomial of X X^T, built up first and applied once: every factor
    # commutes with the others, so the products of a step are those of small matrices
    a, b, c = COEFFICIENTS
    m = s["m"].double() * MU + s["g"].double()
    new = []
    for u, p in zip(_views(case, s["g"].double() + MU * m), _views(case, s["p"].double())):
        u = u / (torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True) + EPS)
        wide = u if u.shape[1] <= u.shape[2] else u.mT
        gram = wide @ wide.mT
        eye = torch.eye(gram.shape[1], dtype=torch.float64, device=gram.device)
        total = eye
        for _ in range(STEPS):
            q = a * eye + gram @ (b * eye + c * gram)
            total, gram = q @ total, q @ gram @ q
        x = total @ wide
        x = x if u.shape[1] <= u.shape[2] else x.mT
        new.append(((1 - LR * WD) * p - LR * math.sqrt(max(1.0, p.shape[1] / p.shape[2])) * x).flatten())
    p = torch.cat(new)
    return {"p": p, "copy": p if case["copy"] else None, "m": m}


def exact(case, seed):
    """What run() gives for these inputs, from the definitions in 64 bits."""
    s = prepare(case, seed)
    return _exact_muon(case, s) if case["op"] == "muon" else _exact_experts(case, s)
