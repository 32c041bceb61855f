"""The AdamW kernels against the formulas in 64 bits, on the GPU.

Tolerances count roundings of float32 (half a step, 2^-24) from the formulas;
an 8-bit state's codes and scales have to be equal: they are decided in 64
bits on both sides, so a value would have to lie within 2^-50 of a border to
be held differently.
"""

import math
import sys

import numpy as np
import pytest
import torch

import tree_allreduce_algorithms_amd as ar

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
H = 2.0 ** -24                                    # half a float32 step
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
HYPER = dict(betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


def announce(msg):
    print(f"[gpu-adamw] {msg}", file=sys.__stderr__, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ar.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def up(x, dtype, offset=0):
    """A device tensor of these values, `offset` elements into its storage."""
    x = torch.as_tensor(np.asarray(x))
    room = torch.zeros(x.numel() + offset, dtype=dtype, device=DEV)
    room[offset:].copy_(x)
    return room[offset:]


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


# --- the definition in 64 bits ---------------------------------------------------

def code_m(m):
    """(codes, scale) of one block, by search among all codes' borders."""
    top = np.max(np.abs(m))
    a = np.float32(top / 127.0 ** 2)
    if not np.isfinite(a):
        return np.zeros(len(m), np.int8), np.float32(np.nan)
    if a == 0:
        return np.zeros(len(m), np.int8), a
    sq = np.arange(128, dtype=np.float64) ** 2
    borders = (sq[1:] + sq[:-1]) / 2
    q = np.searchsorted(borders, np.abs(m) / np.float64(a), side="left")
    return (np.sign(m) * q).astype(np.int8), a


def code_v(v):
    top = np.sqrt(np.max(v))
    r = np.float32(top / 255.0 ** 2)
    if not np.isfinite(r):
        return np.zeros(len(v), np.uint8), np.float32(np.nan)
    if r == 0:
        return np.zeros(len(v), np.uint8), r
    sq = np.arange(256, dtype=np.float64) ** 2
    borders = (sq[1:] + sq[:-1]) / 2
    u = np.searchsorted(borders, np.sqrt(v) / np.float64(r), side="left")
    return np.where(v > 0, np.maximum(u, 1), 0).astype(np.uint8), r


def by_block(fn, x):
    parts = [fn(x[i:i + 256]) for i in range(0, len(x), 256)]
    return np.concatenate([p[0] for p in parts]), np.array([p[1] for p in parts], np.float32)


def scale_of(s, n):
    return np.repeat(s.astype(np.float64), 256)[:n]


def held(st, bits, i):
    """m and v of tensor i as float64, from a host copy of the state."""
    m, v = st["exp_avg"][i], st["exp_avg_sq"][i]
    if bits == 32:
        return m.astype(np.float64), v.astype(np.float64)
    m, v = m.astype(np.float64), v.astype(np.float64)
    n = len(m)
    return (m * np.abs(m) * scale_of(st["exp_avg_scale"][i], n),
            (v * v * scale_of(st["exp_avg_sq_scale"][i], n)) ** 2)


def factor_of(grads, max_norm, grad_scale):
    """(norm in 64 bits, the float32 factor on the gradients)."""
    norm = abs(grad_scale) * math.sqrt(math.fsum(float(x) * float(x) for g in grads for x in g))
    c = np.float32(1.0 if max_norm is None or not norm > max_norm else max_norm / norm)
    return norm, np.float64(np.float32(np.float64(c) * grad_scale))


def step64(p, g, m, v, f, lr, t, betas, eps, weight_decay):
    b1, b2 = betas
    x = g * f
    m1, v1 = b1 * m + (1 - b1) * x, b2 * v + (1 - b2) * x * x
    bc1, bc2 = 1 - b1 ** t, 1 - b2 ** t
    den = np.sqrt(v1 / bc2) + eps
    u = (m1 / bc1) / den
    p1 = p - lr * (weight_decay * p + u)
    # roundings of a float32 evaluation: constant, product(s), sum
    dm = 5 * H * (np.abs(b1 * m) + np.abs((1 - b1) * x)) + 2.0 ** -149
    dv = 7 * H * (np.abs(b2 * v) + (1 - b2) * x * x) + 2.0 ** -149
    return m1, v1, p1, dm, dv, u, den


def param_bound(p, p1, m1, v1, dm, dv, u, den, lr, t, betas, eps, weight_decay, dtype):
    """How far float32 arithmetic on m and v off by dm and dv may leave p'."""
    bc1, bc2 = 1 - betas[0] ** t, 1 - betas[1] ** t
    root = np.sqrt(v1 / bc2)
    droot = np.where(v1 > 0, dv / bc2 / (2 * np.maximum(root, 1e-300)), 0) + np.sqrt(2.0 ** -149 / bc2)
    du = dm / bc1 / den + np.abs(u) * (droot / den + 8 * H)
    dp = lr * du + 4 * H * lr * (np.abs(u) + weight_decay * np.abs(p)) + H * np.abs(p1)
    return dp + (HALF[dtype] * (np.abs(p1) + dp) if dtype != F32 else 0)


SIZES = {"one": [1], "short blocks": [255, 256, 257], "with empty": [0, 1000, 3, 0, 5000],
         "steps": [1023, 1024, 1025, 4096, 4097], "odd": [10_007]}


def make(sizes, bits, pd, gd, copy, offset, seed, spread=True):
    rng = np.random.default_rng(seed)
    p = [up(rng.normal(0, 0.02, n), pd, offset) for n in sizes]
    # gradients over several orders of magnitude
    g = [up(rng.normal(0, 1, n) * 10.0 ** rng.uniform(-6, 0, n) if spread else rng.normal(0, 1, n),
            gd, offset) for n in sizes]
    copies = [up(np.zeros(n), BF16, offset) for n in sizes] if copy else None
    m = [rng.normal(0, 1e-2, n) for n in sizes]
    v = [rng.uniform(0, 1e-2, n) ** 2 for n in sizes]
    if bits == 32:
        state = {"exp_avg": [up(x, F32, offset) for x in m], "exp_avg_sq": [up(x, F32, offset) for x in v]}
    else:
        cm = [by_block(code_m, x) if len(x) else (np.zeros(0, np.int8), np.zeros(0, np.float32)) for x in m]
        cv = [by_block(code_v, x) if len(x) else (np.zeros(0, np.uint8), np.zeros(0, np.float32)) for x in v]
        state = {"exp_avg": [up(x[0], torch.int8, offset) for x in cm],
                 "exp_avg_scale": [up(x[1], F32, offset) for x in cm],
                 "exp_avg_sq": [up(x[0], torch.uint8, offset) for x in cv],
                 "exp_avg_sq_scale": [up(x[1], F32, offset) for x in cv]}
    return p, g, copies, state


def host(state):
    return {k: [t.cpu().numpy().copy() for t in ts] for k, ts in state.items()}


def check_step(opt, bits, lr, max_norm, grad_scale=1.0):
    """One step of `opt`, every output against the definition."""
    before, t = host(opt.state), opt.steps + 1
    p0, g0 = [f64(x) for x in opt.params], [f64(x) for x in opt.grads]
    norm, f = factor_of(g0, max_norm, grad_scale)
    got = opt.grad_norm(max_norm=max_norm)
    opt.step(lr, clip=max_norm is not None)
    torch.cuda.synchronize()
    assert abs(float(got) - norm) <= (H + 1e-12) * norm
    after = host(opt.state)
    for i, n in enumerate(len(x) for x in p0):
        if n == 0:
            continue
        m, v = held(before, bits, i)
        m1, v1, p1, dm, dv, u, den = step64(p0[i], g0[i], m, v, f, lr, t, **HYPER)
        if bits == 32:
            assert np.all(np.abs(after["exp_avg"][i] - m1) <= dm), i
            assert np.all(np.abs(after["exp_avg_sq"][i] - v1) <= dv), i
        else:
            for fn, x, key in ((code_m, m1, "exp_avg"), (code_v, v1, "exp_avg_sq")):
                codes, scales = by_block(fn, x)
                assert np.array_equal(after[key + "_scale"][i], scales), (key, i)
                assert np.array_equal(after[key][i], codes), (key, i)
            # the update takes m' and v' rounded once to float32
            dm, dv = H * np.abs(m1) + 2.0 ** -149, H * v1 + 2.0 ** -149
        out = f64(opt.params[i])
        dp = param_bound(p0[i], p1, m1, v1, dm, dv, u, den, lr, t, dtype=opt.params[i].dtype, **HYPER)
        assert np.all(np.abs(out - p1) <= dp), (i, np.max(np.abs(out - p1) / dp))
        if opt.copies is not None:
            # the copy is the unrounded float32 result's, which is the param itself
            assert torch.equal(opt.copies[i], opt.params[i].to(BF16))


@pytest.mark.parametrize("kind", ["f32 f32", "f32 bf16", "f32 f32 copy", "f32 bf16 copy",
                                  "bf16 f32", "bf16 bf16"])
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_match_the_definition(bits, sizes, offset, kind):
    announce(f"steps {bits} {sizes} {offset} {kind}")
    dt = {"f32": F32, "bf16": BF16}
    pd, gd = (dt[k] for k in kind.split()[:2])
    p, g, copies, state = make(SIZES[sizes], bits, pd, gd, kind.endswith("copy"), offset, 7)
    opt = ar.AdamW(p, g, copies, state_bits=bits, state=state, steps=10, **HYPER)
    for lr, max_norm in ((1e-3, 1.0), (1e-2, None), (1e-3, 1e-3)):
        check_step(opt, bits, lr, max_norm)
    assert opt.steps == 13


@pytest.mark.parametrize("bits", [32, 8])
def test_from_nothing_with_a_gradient_scale(bits):
    """States that start at zero, first steps, gradients that are sums over 8 ranks."""
    p, g, _, _ = make([300, 2000], bits, F32, F32, False, 0, 3)
    opt = ar.AdamW(p, g, state_bits=bits, grad_scale=0.125, **HYPER)
    for max_norm in (0.5, None):
        check_step(opt, bits, 1e-3, max_norm, grad_scale=0.125)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_tiny_and_large_gradients(bits):
    """Blocks of zeros (scale 0, code 0), of subnormal numbers and of 1e15."""
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, 256 * 6)
    x[:256] = 0
    x[256:512] *= 1e-39
    x[512:768] *= 1e-20
    x[768:1024] *= 1e15
    x[1024:1280] = 0.25
    x[1300] = 0
    opt = ar.AdamW([up(rng.normal(0, 0.02, x.size), F32)], [up(x, F32)], state_bits=bits, **HYPER)
    for _ in range(2):
        check_step(opt, bits, 1e-3, None)
    if bits == 8:
        assert float(opt.state["exp_avg_scale"][0][0]) == 0 and not opt.state["exp_avg"][0][:256].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_value_that_is_not_finite_stays_in_its_block(bits, bad):
    p, g, _, state = make([256 * 4 + 7], bits, F32, F32, False, 0, 5)
    hit = 256 + 11
    g[0][hit] = bad
    q, h = [p[0].clone()], [g[0].clone()]
    h[0][hit] = 0
    twin = {k: [t.clone() for t in ts] for k, ts in state.items()}
    opt = ar.AdamW(p, g, state_bits=bits, state=state, **HYPER)
    ref = ar.AdamW(q, h, state_bits=bits, state=twin, **HYPER)
    assert not math.isfinite(float(opt.grad_norm()))
    opt.step(1e-3)
    ref.step(1e-3)
    keep = torch.ones(p[0].numel(), dtype=torch.bool, device=DEV)
    keep[hit] = False
    assert torch.equal(p[0][keep], q[0][keep])
    if bits == 8:
        for k, kind in (("exp_avg", "m"), ("exp_avg_sq", "v")):
            x = ar.dequantize(opt.state[k][0], opt.state[k + "_scale"][0])
            y = ar.dequantize(ref.state[k][0], ref.state[k + "_scale"][0])
            assert torch.isnan(x[256:512]).all()
            assert torch.equal(x[:256], y[:256]) and torch.equal(x[512:], y[512:])
    else:
        assert torch.equal(opt.state["exp_avg"][0][keep], ref.state["exp_avg"][0][keep])


@pytest.mark.parametrize("n", [1, 4097, 3_000_001])
def test_norm_is_the_same_every_time(n):
    g = torch.randn(n, device=DEV)
    opt = ar.AdamW([torch.zeros(n, device=DEV)], [g])
    want = math.sqrt(float(g.double().square().sum()))
    first = opt.grad_norm().clone()
    assert abs(float(first) - want) <= (H + 1e-12) * want
    for _ in range(5):
        assert torch.equal(opt.grad_norm(), first)


@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8])
@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("n", [1, 255, 256 * 256, 256 * 256 + 17])
def test_dequantize_rounds_once(dtype, offset, n):
    rng = np.random.default_rng(9)
    codes = up(np.arange(n) % 256 - (128 if dtype == torch.int8 else 0), dtype, offset)
    scales = up(10.0 ** rng.uniform(-12, 3, -(-n // 256)), F32, offset)
    scales[0] = 0.0 if n > 256 else 1.0
    got = ar.dequantize(codes, scales)
    q, s = f64(codes), scale_of(scales.cpu().numpy(), n)
    want = q * np.abs(q) * s if dtype == torch.int8 else (q * q * s) ** 2
    assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))


def test_dequantize_of_nothing():
    got = ar.dequantize(torch.zeros(0, dtype=torch.int8, device=DEV), torch.zeros(0, device=DEV))
    assert got.shape == (0,) and got.dtype == F32


def test_refusals():
    x, y = torch.zeros(8, device=DEV), torch.zeros(8, device=DEV)
    h = torch.zeros(8, device=DEV, dtype=BF16)
    bad = [(ValueError, dict(params=[x], grads=[])), (ValueError, dict(params=[x], grads=[y[:4]])),
           (TypeError, dict(params=[x], grads=[y.int()])), (TypeError, dict(params=[x, h], grads=[y, y])),
           (ValueError, dict(params=[x], grads=[torch.zeros(16, device=DEV)[::2]])),
           (TypeError, dict(params=[h], grads=[y], copies=[h.clone()])),
           (ValueError, dict(params=[x], grads=[y], state_bits=16)),
           (ValueError, dict(params=[x], grads=[y], steps=-1)),
           (ValueError, dict(params=[x], grads=[y], state={"exp_avg": [x]})),
           (ar.ArError, dict(params=[x], grads=[x])),                     # over each other
           (ar.ArError, dict(params=[x, x], grads=[y, y]))]
    for error, kw in bad:
        with pytest.raises(error):
            ar.AdamW(**kw)
    opt = ar.AdamW([x], [y])
    with pytest.raises(ValueError, match="clip"):
        opt.step(1e-3, clip=True)
    opt.grad_norm()                                                    # no bound was given
    with pytest.raises(ValueError, match="clip"):
        opt.step(1e-3, clip=True)
    opt.grad_norm(max_norm=1.0)
    opt.step(1e-3, clip=True)
    with pytest.raises(ValueError, match="clip"):                      # the gradients' norm before
        opt.step(1e-3, clip=True)
    for lr in (-1.0, float("nan")):
        with pytest.raises(ar.ArError):
            opt.step(lr)
    with pytest.raises(ar.ArError):
        opt.grad_norm(max_norm=-1.0)
    assert opt.steps == 1
    ar.debug_fail_launch(1)
    with pytest.raises(ar.ArError):
        opt.step(1e-3)
    assert opt.steps == 1
    codes = torch.zeros(300, dtype=torch.int8, device=DEV)
    for error, args in ((TypeError, (codes.int(), x)), (ValueError, (codes, x)),
                        (ValueError, (codes[::2], x[:1])), (TypeError, (codes, x[:2].double()))):
        with pytest.raises(error):
            ar.dequantize(*args)


def test_side_stream_and_graph():
    """Steps on a side stream equal those on the default one; a captured norm
    follows the gradients from replay to replay; a step refuses capture."""
    p, g, _, state = make([5000, 300], 8, F32, F32, False, 0, 21)
    q = [t.clone() for t in p]
    twin = {k: [t.clone() for t in ts] for k, ts in state.items()}
    a = ar.AdamW(p, g, state_bits=8, state=state)
    b = ar.AdamW(q, g, state_bits=8, state=twin)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.grad_norm(max_norm=1.0)
        a.step(1e-3, clip=True)
        b.grad_norm(max_norm=1.0, stream=side)
        b.step(1e-3, clip=True, stream=side)
    x = ar.dequantize(b.state["exp_avg"][0], b.state["exp_avg_scale"][0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(s, t) for s, t in zip(p, q))
    assert torch.equal(x, ar.dequantize(a.state["exp_avg"][0], a.state["exp_avg_scale"][0]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = a.grad_norm(max_norm=1.0)
        with pytest.raises(ar.ArError, match="unsupported"):
            a.step(1e-3, clip=True)
    for k in range(4):
        for t in g:
            t.normal_()
        want = math.sqrt(sum(float(t.double().square().sum()) for t in g))
        graph.replay()
        torch.cuda.synchronize()
        assert abs(float(norm) - want) <= (H + 1e-12) * want, k


def test_offsets_past_32_bits():
    """One tensor of 2^32 + 1,000 elements: its end is computed as its start is."""
    n, tail = (1 << 32) + 1000, 3000
    p = torch.zeros(n, dtype=BF16, device=DEV)
    g = torch.zeros(n, dtype=BF16, device=DEV)
    p[-tail:].normal_(0, 0.02)
    g[-tail:].normal_(0, 1)
    opt = ar.AdamW([p], [g], state_bits=8, **HYPER)
    # the same values as a small tensor whose blocks begin at the same places
    begin = (n - tail) // 256 * 256
    q, h = p[begin:].clone(), g[begin:].clone()
    ref = ar.AdamW([q], [h], state_bits=8, **HYPER)
    for o in (opt, ref):
        o.step(1e-3)
    assert torch.equal(p[begin:], q) and not p[:1000].any()
    assert torch.equal(opt.state["exp_avg"][0][begin:], ref.state["exp_avg"][0])
    assert torch.equal(opt.state["exp_avg_sq_scale"][0][begin // 256:], ref.state["exp_avg_sq_scale"][0])
    assert float(opt.grad_norm()) == float(ref.grad_norm())
    x = ar.dequantize(opt.state["exp_avg"][0], opt.state["exp_avg_scale"][0])
    assert torch.equal(x[begin:], ar.dequantize(ref.state["exp_avg"][0], ref.state["exp_avg_scale"][0]))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_small_problem_is_solved(bits):
    """Least squares: both kinds of state reach the solution."""
    torch.manual_seed(0)
    target = torch.randn(1000, device=DEV)
    w, g = torch.zeros(1000, device=DEV), torch.zeros(1000, device=DEV)
    opt = ar.AdamW([w], [g], state_bits=bits, weight_decay=0.0)
    for k in range(300):
        torch.sub(w, target, out=g)
        opt.grad_norm(max_norm=1.0)
        opt.step(0.05 * (1 - k / 300), clip=True)
    assert float((w - target).abs().max()) < 0.05
