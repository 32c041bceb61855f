"""The experts' products against the definition in 64 bits, on the GPU.

Orders have to be equal.  A product's element is a float32 sum of exact
products (bfloat16 times bfloat16 fits float32) in some order: off by at most n
steps of float32 (2^-23, whether an addition rounds or cuts) of the sum of the
products' sizes, and then half a step of bfloat16 (2^-8) where it is stored so.
"""

import sys

import numpy as np
import pytest
import torch

import tree_allreduce_algorithms_amd as ar

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
HALF = 2.0 ** -8          # half a step of bfloat16, relative
STEP = 2.0 ** -23
TINY = 2.0 ** -126


def announce(msg):
    print(f"[gpu-experts] {msg}", file=sys.__stderr__, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ar.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def choices(tokens, k, experts, kind, seed):
    """[tokens, k] int32 on the CPU."""
    rng = np.random.default_rng(seed)
    if kind == "one":                       # every pair to one expert
        return np.full((tokens, k), experts - 1, np.int32)
    if kind == "none":
        return np.full((tokens, k), -1, np.int32)
    skew = rng.permutation(experts) + 1.0 if kind == "skewed" else np.ones(experts)
    p = (1 / skew) / (1 / skew).sum()
    x = rng.choice(experts, (tokens, k), p=p).astype(np.int32)
    if kind == "masked":
        x[rng.random(tokens) < 0.3] = -1
        x[rng.random((tokens, k)) < 0.1] = -1
    return x


def order_of(x, experts):
    """(order, position, offsets) by the definition."""
    flat = x.reshape(-1)
    live = (flat >= 0) & (flat < experts)
    key = np.where(live, flat, experts)
    order = np.argsort(key, kind="stable")[:live.sum()].astype(np.int32)
    position = np.full(flat.size, -1, np.int32)
    position[order] = np.arange(order.size)
    offsets = np.searchsorted(key[order], np.arange(experts + 1)).astype(np.int32)
    return np.concatenate([order, np.full(flat.size - order.size, -1, np.int32)]), position, offsets


def bf16(rng, *shape, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * scale).to(DEV).to(BF16)


def grouped(x, w, order, offsets, k, gather):
    """Rows in float64 and the sums of the products' sizes."""
    pairs, experts = order.size, offsets.size - 1
    y = torch.zeros(pairs, w.shape[2], dtype=torch.float64, device=DEV)
    size = torch.zeros_like(y)
    o = torch.from_numpy(order.astype(np.int64)).to(DEV)
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo < hi:
            rows = x[o[lo:hi] // k] if gather else x[lo:hi]
            y[lo:hi] = rows.double() @ w[e].double()
            size[lo:hi] = rows.double().abs() @ w[e].double().abs()
    return y, size


def near(got, want, size, n, what, stored=True):
    bound = n * STEP * size + TINY
    if stored:
        bound = bound + HALF * (want.abs() + bound)
    off = (got.double() - want).abs()
    worst = float((off / bound).max()) if off.numel() else 0.0
    assert bool((off <= bound).all()), f"{what}: {worst:.2f} of the bound"


# --- order -----------------------------------------------------------------------

@pytest.mark.parametrize("tokens,k,experts,kind", [
    (1, 1, 1, "even"), (1, 8, 8, "even"), (1, 2, 1024, "even"), (5, 3, 7, "masked"), (63, 1, 64, "skewed"),
    (1000, 4, 61, "masked"), (512, 8, 256, "skewed"), (4096, 1, 3, "one"), (700, 2, 16, "none"),
    (1024, 1, 5, "masked"), (1025, 1, 5, "skewed"), (32768, 1, 1024, "masked"), (32769, 1, 9, "masked"),
    (16384, 8, 1024, "skewed"), (16384, 8, 128, "masked"), (40000, 6, 64, "even"), (12289, 1, 1000, "masked"),
])
def test_order(tokens, k, experts, kind):
    announce(f"order {tokens} {k} {experts} {kind}")
    x = choices(tokens, k, experts, kind, tokens + k)
    o = ar.expert_order(torch.from_numpy(x).to(DEV), experts)
    order, position, offsets = order_of(x, experts)
    assert np.array_equal(o.offsets.cpu().numpy(), offsets)
    assert np.array_equal(o.order.cpu().numpy(), order)
    assert o.position.shape == (tokens, k)
    assert np.array_equal(o.position.cpu().numpy().reshape(-1), position)


def test_order_of_no_pairs_and_of_numbers_that_are_no_experts():
    o = ar.expert_order(torch.zeros(0, 4, dtype=torch.int32, device=DEV), 5)
    assert o.order.numel() == 0 and o.position.shape == (0, 4) and o.offsets.tolist() == [0] * 6
    wild = torch.tensor([[3, -1, 4], [2 ** 31 - 1, -2 ** 31, 0]], dtype=torch.int32, device=DEV)
    o = ar.expert_order(wild, 4)
    assert o.order.tolist() == [5, 0, -1, -1, -1, -1] and o.offsets.tolist() == [0, 1, 1, 1, 2]
    assert o.position.tolist() == [[1, -1, -1], [-1, -1, 0]]


# --- products ----------------------------------------------------------------------

SHAPES = [
    # tokens, top_k, experts, in, out, kind
    (1, 2, 8, 64, 64, "even"), (1, 1, 1, 1, 1, "even"), (3, 2, 4, 7, 5, "masked"), (40, 4, 61, 72, 136, "masked"),
    (130, 1, 1, 200, 129, "even"), (129, 2, 3, 64, 128, "one"), (64, 8, 16, 1000, 24, "skewed"),
    (300, 2, 5, 33, 300, "skewed"), (257, 3, 1000, 65, 66, "masked"), (20, 2, 4, 128, 256, "none"),
    (3000, 2, 40, 128, 264, "skewed"), (2000, 2, 8, 256, 512, "skewed"), (513, 8, 64, 520, 392, "masked"), (7, 2, 8, 2048, 1024, "even"),
]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("tokens,k,experts,n_in,n_out,kind", SHAPES)
def test_matmul(tokens, k, experts, n_in, n_out, kind, turned, gather):
    announce(f"matmul {tokens} {k} {experts} {n_in} {n_out} {kind} turned={turned} gather={gather}")
    rng = np.random.default_rng(n_in * 31 + n_out)
    idx = choices(tokens, k, experts, kind, 5)
    order, _, offsets = order_of(idx, experts)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), experts)
    x = bf16(rng, tokens if gather else tokens * k, n_in)
    w = bf16(rng, experts, n_out, n_in).transpose(1, 2) if turned else bf16(rng, experts, n_in, n_out)
    y = ar.expert_matmul(x, w, o, gather=gather)
    want, size = grouped(x, w, order, offsets, k, gather)
    assert y.shape == want.shape and y.dtype == BF16
    near(y, want, size, n_in, "y")
    assert not y[int(offsets[-1]):].any()


@pytest.mark.parametrize("cut", ["rows apart", "odd rows", "odd address", "weights apart", "expert strides"])
@pytest.mark.parametrize("turned", [False, True])
def test_matmul_of_views(turned, cut):
    """Rows, columns and experts cut out of larger tensors, at any element."""
    announce(f"views {cut} turned={turned}")
    rng = np.random.default_rng(3)
    tokens, k, experts, n_in, n_out = 150, 2, 5, 96, 160
    idx = choices(tokens, k, experts, "masked", 1)
    order, _, offsets = order_of(idx, experts)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), experts)
    x, w = bf16(rng, tokens, n_in), bf16(rng, experts, n_in, n_out)
    if turned:
        w = w.transpose(1, 2).contiguous().transpose(1, 2)
    want, size = grouped(x, w, order, offsets, k, True)
    if cut == "rows apart":
        x = torch.full((tokens, n_in + 40), float("nan"), dtype=BF16, device=DEV)[:, 8:8 + n_in].copy_(x)
    elif cut == "odd rows":
        x = torch.full((tokens, n_in + 1), float("nan"), dtype=BF16, device=DEV)[:, :n_in].copy_(x)
    elif cut == "odd address":
        flat = torch.full((x.numel() + 3,), float("nan"), dtype=BF16, device=DEV)
        x = flat[3:].view(tokens, n_in).copy_(x)
    elif cut == "weights apart":
        big = torch.full((experts, n_in + 24, n_out + 24), float("nan"), dtype=BF16, device=DEV)
        if turned:
            big = big.transpose(1, 2).contiguous().transpose(1, 2)
        w = big[:, 16:16 + n_in, 8:8 + n_out].copy_(w)
    else:
        big = torch.full((2 * experts, n_in, n_out), float("nan"), dtype=BF16, device=DEV)
        if turned:
            big = big.transpose(1, 2).contiguous().transpose(1, 2)
        w = big[1::2].copy_(w)
    near(ar.expert_matmul(x, w, o, gather=True), want, size, n_in, cut)
    shared = w[:1].expand(experts, -1, -1)      # one matrix for all
    want, size = grouped(x, shared, order, offsets, k, True)
    near(ar.expert_matmul(x, shared, o, gather=True), want, size, n_in, "shared")


@pytest.mark.parametrize("sizes", [(96, 160), (61, 77)])
def test_values_stay_in_their_rows(sizes):
    """A row or an expert that is not finite shows in its own results alone, padding shows nowhere."""
    rng = np.random.default_rng(4)
    tokens, k, experts, (n_in, n_out) = 90, 2, 4, sizes
    idx = choices(tokens, k, experts, "masked", 2)
    idx[7] = [1, 2]
    order, _, offsets = order_of(idx, experts)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), experts)
    x, w = bf16(rng, tokens, n_in), bf16(rng, experts, n_in, n_out)
    clean = ar.expert_matmul(x, w, o, gather=True)
    x[7], w[3] = float("nan"), float("inf")
    y = ar.expert_matmul(x, w, o, gather=True)
    pairs = torch.from_numpy(order.astype(np.int64)).to(DEV)
    rows = torch.arange(order.size, device=DEV)
    live = rows < int(offsets[-1])
    of_token = live & (pairs // k == 7)
    of_expert = live & (rows >= int(offsets[3])) & (rows < int(offsets[4]))
    assert bool(y[of_token].isnan().all()) and int(of_token.sum()) == 2
    assert not bool(y[of_expert].isfinite().any())
    rest = ~(of_token | of_expert)
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("tokens,k,experts,n_in,n_out,kind", SHAPES)
def test_weight_grad(tokens, k, experts, n_in, n_out, kind, gather, dtype):
    announce(f"weight_grad {tokens} {k} {experts} {n_in} {n_out} {kind} gather={gather} {dtype}")
    rng = np.random.default_rng(n_in * 37 + n_out)
    idx = choices(tokens, k, experts, kind, 6)
    order, _, offsets = order_of(idx, experts)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), experts)
    x, dy = bf16(rng, tokens if gather else tokens * k, n_in), bf16(rng, tokens * k, n_out)
    dy[int(offsets[-1]):] = float("nan")       # rows without an expert are not read
    dw = ar.expert_weight_grad(x, dy, o, gather=gather, dtype=dtype)
    assert dw.shape == (experts, n_in, n_out) and dw.dtype == dtype
    rows = torch.from_numpy(order.astype(np.int64)).to(DEV)
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        xs = (x[rows[lo:hi] // k] if gather else x[lo:hi]).double().t().contiguous()
        d = dy[lo:hi].double()
        near(dw[e], xs @ d, xs.abs() @ d.abs(), max(1, hi - lo), f"dw {e}", stored=dtype == BF16)


@pytest.mark.parametrize("tokens,k,experts,n_in,n_out,kind", [
    (5000, 1, 1, 64, 96, "even"), (3001, 2, 2, 130, 264, "skewed"), (2000, 3, 4, 61, 77, "masked"), (8000, 1, 5, 64, 64, "skewed"), (4000, 1, 3, 40, 8, "one"),
])
def test_weight_grad_of_shared_rows(tokens, k, experts, n_in, n_out, kind):
    """Few tiles: several blocks share an expert's rows."""
    assert ar.lib().ar_expert_weight_grad_workspace(tokens * k, experts, n_in, n_out) > 0
    for gather, dtype in ((True, F32), (False, BF16), (True, BF16)):
        test_weight_grad(tokens, k, experts, n_in, n_out, kind, gather, dtype)


def test_weight_grad_into_a_tensor():
    rng = np.random.default_rng(5)
    idx = choices(100, 2, 6, "even", 3)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), 6)
    x, dy = bf16(rng, 100, 40), bf16(rng, 200, 24)
    want = ar.expert_weight_grad(x, dy, o, gather=True)
    flat = torch.full((6 * 40 * 24 + 10,), float("nan"), device=DEV)
    out = flat[5:-5].view(6, 40, 24)
    before = out._version
    assert ar.expert_weight_grad(x, dy, o, gather=True, out=out) is out
    assert torch.equal(out, want) and out._version > before
    assert bool(flat[:5].isnan().all() and flat[-5:].isnan().all())


# --- sums ---------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,k,experts,size,kind", [
    (1, 1, 1, 1, "even"), (1, 8, 8, 1024, "even"), (33, 3, 7, 61, "masked"), (5, 2, 4, 4096, "masked"),
    (1000, 4, 16, 520, "masked"), (64, 2, 4, 128, "none"), (300, 6, 64, 2049, "skewed"),
    (100, 2, 8, 7, "even"), (100, 2, 8, 9, "masked"), (50, 4, 8, 515, "even"), (40, 3, 8, 1030, "masked"),
    (8200, 4, 8, 1026, "masked"), (16400, 8, 8, 520, "even"), (8200, 2, 8, 1024, "masked"),
])
def test_combine_and_its_gradient(tokens, k, experts, size, kind):
    announce(f"combine {tokens} {k} {experts} {size} {kind}")
    rng = np.random.default_rng(size)
    idx = choices(tokens, k, experts, kind, 8)
    _, position, offsets = order_of(idx, experts)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), experts)
    y = bf16(rng, tokens * k, size)
    w = torch.from_numpy(rng.random((tokens, k)).astype(np.float32)).to(DEV)
    y[int(offsets[-1]):] = float("nan")
    pos = torch.from_numpy(position.astype(np.int64)).to(DEV).view(tokens, k)
    chosen = (pos >= 0)[..., None]
    rows = torch.where(chosen, y.double()[pos], 0.0)
    # without a row the weight is not looked at either
    wild = torch.where(chosen[..., 0], w, float("nan"))
    for weights in (None, wild):
        one = torch.ones_like(w) if weights is None else w
        terms = one.double()[..., None] * rows
        near(ar.expert_combine(y, o, weights), terms.sum(1), terms.abs().sum(1), k, "out")

    dout = bf16(rng, tokens, size)
    dy, dw = ar.expert_combine_grad(dout, y, o, wild)
    want = torch.zeros(tokens * k, size, dtype=torch.float64, device=DEV)
    want[pos[chosen[..., 0]]] = (w.double()[..., None] * dout.double()[:, None])[chosen[..., 0]]
    near(dy, want, want.abs(), 1, "dy")
    terms = dout.double()[:, None] * rows
    near(dw, terms.sum(-1), terms.abs().sum(-1), size, "dweights", stored=False)
    assert dw.shape == (tokens, k) and not dw[~chosen[..., 0]].any()


def test_sums_of_views():
    rng = np.random.default_rng(9)
    idx = choices(70, 3, 5, "masked", 9)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), 5)
    y, dout = bf16(rng, 210, 50), bf16(rng, 70, 50)
    w = torch.rand(70, 3, device=DEV)
    cut = lambda t: torch.full((t.shape[0], 61), float("nan"), dtype=BF16, device=DEV)[:, 3:53].copy_(t)  # noqa: E731
    assert torch.equal(ar.expert_combine(y, o, w), ar.expert_combine(cut(y), o, w))
    for a, b in zip(ar.expert_combine_grad(dout, y, o, w), ar.expert_combine_grad(cut(dout), cut(y), o, w)):
        assert torch.equal(a, b)


# --- the ends of the ranges ---------------------------------------------------------

def test_no_tokens():
    o = ar.expert_order(torch.zeros(0, 4, dtype=torch.int32, device=DEV), 5)
    x, w = torch.empty(0, 24, dtype=BF16, device=DEV), torch.randn(5, 24, 32, device=DEV).to(BF16)
    y = ar.expert_matmul(x, w, o, gather=True)
    assert y.shape == (0, 32) and ar.expert_matmul(x, w, o).shape == (0, 32)
    g = torch.empty(0, 4, device=DEV)
    assert ar.expert_combine(y, o, g).shape == (0, 32)
    dy, dg = ar.expert_combine_grad(torch.empty(0, 32, dtype=BF16, device=DEV), y, o, g)
    assert dy.shape == (0, 32) and dg.shape == (0, 4)
    dw = ar.expert_weight_grad(x, dy, o, gather=True)
    assert dw.shape == (5, 24, 32) and not dw.any()


def test_many_choices_of_few_tokens():
    """pairs * top_k past 32 bits: a pair's token by division."""
    idx = choices(3, 60_000, 7, "even", 4)
    order, _, offsets = order_of(idx, 7)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), 7)
    rng = np.random.default_rng(6)
    x, w = bf16(rng, 3, 16), bf16(rng, 7, 16, 8)
    want, size = grouped(x, w, order, offsets, 60_000, True)
    near(ar.expert_matmul(x, w, o, gather=True), want, size, 16, "y")
    dy = bf16(rng, 180_000, 8)
    dw = ar.expert_weight_grad(x, dy, o, gather=True)
    token = torch.from_numpy(order.astype(np.int64)).to(DEV) // 60_000
    for e in range(7):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        xs, d = x[token[lo:hi]].double().t().contiguous(), dy[lo:hi].double()
        near(dw[e], xs @ d, xs.abs() @ d.abs(), hi - lo, f"dw {e}", stored=False)


@pytest.mark.parametrize("n_in", [64, 61])
def test_rows_past_32_bits(n_in):
    """x's and dy's rows beyond 4 GiB from their beginning, y's too."""
    tokens, k, experts, n_out, far = 40_000, 2, 3, 32_768, 65_536
    idx = choices(tokens, k, experts, "even", 7)
    order, _, offsets = order_of(idx, experts)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), experts)
    rng = np.random.default_rng(8)
    small = bf16(rng, tokens, n_in)
    x = torch.zeros(tokens, far, dtype=BF16, device=DEV)[:, :n_in].copy_(small)
    w = bf16(rng, experts, n_in, n_out)
    y = ar.expert_matmul(x, w, o, gather=True)              # 80,000 x 32,768: 5.2 GB
    pairs = torch.from_numpy(order.astype(np.int64)).to(DEV)
    for i in (0, 1, 39_999, 65_536, 79_999):
        e = int(np.searchsorted(offsets, i, side="right")) - 1
        row = small[pairs[i] // k].double()
        near(y[i:i + 1], (row @ w[e].double())[None], (row.abs() @ w[e].double().abs())[None], n_in, f"y {i}")
    out = ar.expert_combine(y, o)
    position = torch.from_numpy(order_of(idx, experts)[1].astype(np.int64)).to(DEV).view(tokens, k)
    for t in (0, 20_000, 39_999):
        rows = y[position[t]].double()
        near(out[t:t + 1], rows.sum(0)[None], rows.abs().sum(0)[None], k, f"out {t}")
    dw = ar.expert_weight_grad(x, y[:, :24], o, gather=True)      # dy's rows 65,536 bytes apart
    lo, hi = int(offsets[2]), int(offsets[3])
    xs, d = small[pairs[lo:hi] // k].double().t().contiguous(), y[lo:hi, :24].double()
    near(dw[2], xs @ d, xs.abs() @ d.abs(), hi - lo, "dw", stored=False)


# --- a layer, as it is used -----------------------------------------------------------

def test_gradients_of_a_layer():
    """Two products and a nonlinearity after the router: the chain of calls against
    autograd of the formula in float64, and one direction against differences."""
    rng = np.random.default_rng(11)
    tokens, k, experts, d, h = 96, 2, 6, 48, 80
    x, w1, w2 = bf16(rng, tokens, d), bf16(rng, experts, d, h, scale=0.15), bf16(rng, experts, h, d, scale=0.1)
    logits = bf16(rng, tokens, experts).float()
    mask = torch.from_numpy(rng.random(tokens) > 0.1).to(DEV)
    r = ar.route([logits], k, mask=[mask], renormalize=True)
    o = ar.expert_order(r.indices, experts)
    u = ar.expert_matmul(x, w1, o, gather=True)
    a = torch.relu(u)
    y = ar.expert_matmul(a, w2, o)
    out = ar.expert_combine(y, o, r.weights)
    dout = bf16(rng, tokens, d)
    dy, dweights = ar.expert_combine_grad(dout, y, o, r.weights)
    dw2 = ar.expert_weight_grad(a, dy, o)
    du = ar.expert_matmul(dy, w2.transpose(1, 2), o) * (u > 0)
    dw1 = ar.expert_weight_grad(x, du, o, gather=True)
    dx = ar.expert_combine(ar.expert_matmul(du, w1.transpose(1, 2), o), o)

    X, W1, W2 = (t.double().requires_grad_() for t in (x, w1, w2))
    gate = r.weights[0].double().requires_grad_()
    index = r.indices[0].long()
    live = (index >= 0)[..., None]

    def layer(X, W1, W2, gate):
        hidden = (X[:, None, :, None] * W1[index.clamp(min=0)]).sum(2)
        rows = (torch.relu(hidden)[..., None] * W2[index.clamp(min=0)]).sum(2)
        return (gate[..., None] * torch.where(live, rows, 0.0)).sum(1)

    want = layer(X, W1, W2, gate)
    want.backward(dout.double())
    # four roundings at most lie between an input and a result, each of half a
    # step of values no larger than the result's terms: 2-norms, with a factor 2 for
    # signs of u that a rounding turns
    for got, exact, roundings, what in ((out, want, 3, "out"), (dweights, gate.grad, 2, "dweights"),
                                        (dw2, W2.grad, 2, "dw2"), (dw1, W1.grad, 3, "dw1"), (dx, X.grad, 4, "dx")):
        off = float((got.double() - exact.detach()).norm() / exact.detach().norm())
        assert off <= 2 * roundings * HALF, f"{what}: {off}"
    # one direction of W1 by differences of the formula
    V = torch.from_numpy(rng.standard_normal(w1.shape)).to(DEV)
    eps = 1e-6
    with torch.no_grad():
        slope = ((layer(X, W1 + eps * V, W2, gate) - layer(X, W1 - eps * V, W2, gate)) * dout.double()).sum() / (2 * eps)
    scale = float((dw1.double() * V).norm())
    assert abs(float((dw1.double() * V).sum()) - float(slope)) <= 2 * 3 * HALF * scale * 3


# --- streams, graphs, refusals -----------------------------------------------------------

def run_all(x, w, idx, weights, dout, experts, stream=None):
    o = ar.expert_order(idx, experts, stream=stream)
    y = ar.expert_matmul(x, w, o, gather=True, stream=stream)
    out = ar.expert_combine(y, o, weights, stream=stream)
    dy, dweights = ar.expert_combine_grad(dout, y, o, weights, stream=stream)
    rows = ar.expert_matmul(dy, w.transpose(1, 2), o, stream=stream)
    dx = ar.expert_combine(rows, o, stream=stream)
    dw = ar.expert_weight_grad(x, dy, o, gather=True, stream=stream)
    return [o.order, o.offsets, y, out, dy, dweights, dx, dw]


def inputs(seed, tokens=300, k=2, experts=8, n_in=128, n_out=192):
    rng = np.random.default_rng(seed)
    return [bf16(rng, tokens, n_in), bf16(rng, experts, n_in, n_out, scale=n_in ** -0.5),
            torch.from_numpy(choices(tokens, k, experts, "masked", seed)).to(DEV),
            torch.rand(tokens, k, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)), bf16(rng, tokens, n_out)]


def test_on_a_named_stream_with_inputs_dropped():
    args = inputs(21, tokens=6000)
    want = run_all(*args, 8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = run_all(*args, 8, stream=side)
    like, used = [torch.empty_like(t) for t in args], {t.data_ptr() for t in args}
    del args
    again = [torch.zeros_like(t) for t in like for _ in range(2)]
    assert not used & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed_beside_eager_calls():
    args, other = inputs(22, tokens=5000), inputs(23, tokens=5000)
    run_all(*args, 8)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        held = run_all(*args, 8)
    for seed in range(3):
        fresh = inputs(30 + seed, tokens=5000)
        for a, b in zip(args, fresh):
            a.copy_(b)
        graph.replay()
        beside = run_all(*other, 8)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, run_all(*fresh, 8))), seed
        assert all(torch.equal(a, b) for a, b in zip(beside, run_all(*other, 8))), seed


def test_the_same_call_gives_the_same_bits():
    args = inputs(24, tokens=4000, experts=16)
    first = run_all(*args, 16)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, run_all(*args, 16)))


def test_refusals():
    x, w, idx, weights, dout = inputs(25)
    o = ar.expert_order(idx, 8)
    y = ar.expert_matmul(x, w, o, gather=True)
    ok = lambda: ar.expert_matmul(x, w, o, gather=True)  # noqa: E731
    bad = [
        (TypeError, lambda: ar.expert_order(idx.cpu(), 8)), (TypeError, lambda: ar.expert_order(idx.long(), 8)),
        (ValueError, lambda: ar.expert_order(idx, 0)), (ValueError, lambda: ar.expert_order(idx, 1025)),
        (ValueError, lambda: ar.expert_order(idx.t(), 8)), (ValueError, lambda: ar.expert_order(idx[0, 0], 8)),
        (ValueError, lambda: ar.expert_order(idx[:, :0], 8)), (TypeError, lambda: ar.expert_order([1, 2], 8)),
        (TypeError, lambda: ar.expert_matmul(x, w, idx)), (TypeError, lambda: ar.expert_matmul(x.float(), w, o)),
        (TypeError, lambda: ar.expert_matmul(x, w.float(), o, gather=True)),
        (TypeError, lambda: ar.expert_matmul(x.cpu(), w, o, gather=True)),
        (TypeError, lambda: ar.expert_matmul(x, w.cpu(), o, gather=True)),
        (ValueError, lambda: ar.expert_matmul(x, w, o)), (ValueError, lambda: ar.expert_matmul(x[:5], w, o, gather=True)),
        (ValueError, lambda: ar.expert_matmul(x, w[:7], o, gather=True)),
        (ValueError, lambda: ar.expert_matmul(x[:, :64], w, o, gather=True)),
        (ValueError, lambda: ar.expert_matmul(x, w[:, :, ::2], o, gather=True)),
        (ValueError, lambda: ar.expert_matmul(x.t().contiguous().t(), w, o, gather=True)),
        (ValueError, lambda: ar.expert_matmul(x[:1].expand(300, -1), w, o, gather=True)),
        (ValueError, lambda: ar.expert_matmul(x[:, :0], w[:, :0], o, gather=True)),
        (ValueError, lambda: ar.expert_weight_grad(x, y[:5], o, gather=True)),
        (TypeError, lambda: ar.expert_weight_grad(x, y.float(), o, gather=True)),
        (TypeError, lambda: ar.expert_weight_grad(x, y, o, gather=True, dtype=torch.float16)),
        (TypeError, lambda: ar.expert_weight_grad(x, y, o, gather=True, out=torch.empty(8, 128, 192, device=DEV).int())),
        (ValueError, lambda: ar.expert_weight_grad(x, y, o, gather=True, out=torch.empty(8, 192, 128, device=DEV))),
        (ValueError, lambda: ar.expert_weight_grad(x, y, o, gather=True,
                                                   out=torch.empty(8, 192, 128, device=DEV).transpose(1, 2))),
        (ValueError, lambda: ar.expert_combine(y[:5], o, weights)), (TypeError, lambda: ar.expert_combine(y.float(), o)),
        (TypeError, lambda: ar.expert_combine(y, o, weights.bfloat16())),
        (ValueError, lambda: ar.expert_combine(y, o, weights[:5])),
        (ValueError, lambda: ar.expert_combine(y, o, weights.t().contiguous().t())),
        (TypeError, lambda: ar.expert_combine_grad(dout, y, o, None)),
        (ValueError, lambda: ar.expert_combine_grad(dout[:, :5], y, o, weights)),
    ]
    ar.debug_fail_launch(1)           # none of them gets as far as a launch
    try:
        for i, (error, call) in enumerate(bad):
            with pytest.raises(error):
                call()
                raise AssertionError(f"case {i} was taken")
        with pytest.raises(ar.ArError):
            ok()
    finally:
        ar.debug_fail_launch(0)
    want = ok()
    # an order's tensors are plain attributes: what the kernels read is checked
    for name, change in (("order", lambda t: t.long()), ("offsets", lambda t: t[:8]), ("position", lambda t: t[:5]),
                         ("offsets", lambda t: t.cpu()), ("top_k", lambda t: 7), ("top_k", lambda t: 0)):
        p = ar.expert_order(idx, 8)
        setattr(p, name, change(getattr(p, name)))
        with pytest.raises((TypeError, ValueError)):
            ar.expert_matmul(x, w, p, gather=True)
    # numbers out of range in them name no row
    p = ar.expert_order(idx, 8)
    p.order = torch.full_like(p.order, 2 ** 31 - 1)
    assert not ar.expert_matmul(x, w, p, gather=True).any()
    assert not ar.expert_weight_grad(x, y, p, gather=True).any()
    p.position = torch.full_like(p.position, 10 ** 6)
    assert not ar.expert_combine(y, p, weights).any()
    p.offsets = torch.tensor([0, 10 ** 9, -5, 7, 2 ** 31 - 1, 0, 1, 2, 3], dtype=torch.int32, device=DEV)
    ar.expert_matmul(x, w, p, gather=True)
    ar.expert_weight_grad(x, y, p, gather=True)
    ar.expert_combine_grad(dout, y, p, weights)
    torch.cuda.synchronize()
    assert torch.equal(ok(), want)
