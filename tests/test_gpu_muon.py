"""The Muon step against its formula in 64 bits, on the GPU.

The Newton-Schulz steps multiply what an earlier step's rounding left by up to
3.9 each (the polynomial's steepest slope), so no useful bound holds for all
matrices; what they make of a matrix is measured instead.  A product here has
operands of 22 bits and float32 sums, so it is off by at most 4 + 1 times what
float32's product is (24 bits, the same sums), and what it leaves goes through
the same steps: the result may be 8 times as far from the formula as that of
float32 products on the CPU (2-norms), and a few roundings (2^-24) beside that.
"""

import sys

import numpy as np
import pytest
import torch

import tree_allreduce_algorithms_amd as ar

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
H = 2.0 ** -24
A, B, C = 3.4445, -4.7750, 2.0315


def announce(msg):
    print(f"[gpu-muon] {msg}", file=sys.__stderr__, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ar.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def orthogonal(u, steps, eps, dtype):
    """[..., rows, cols] on the CPU, products in `dtype`."""
    u = u.double()
    x = (u / (u.square().sum((-2, -1), keepdim=True).sqrt() + eps)).to(dtype)
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-2, -1).contiguous() if tall else x
    for _ in range(steps):
        gram = x @ x.transpose(-2, -1).contiguous()
        x = A * x + (B * gram + C * (gram @ gram)) @ x
    return (x.transpose(-2, -1) if tall else x).double()


def expected(p, g, m, h):
    """(p', m', 2-norm bound of p') of tensors on the CPU."""
    m = h["momentum"] * m.double() + h["grad_scale"] * g.double()
    u = h["grad_scale"] * g.double() + h["momentum"] * m if h["nesterov"] else m
    rows, cols = p.shape[-2:]
    s = max(1.0, rows / cols) ** 0.5 if h["match_rms"] is None else h["match_rms"] * max(rows, cols) ** 0.5
    x = orthogonal(u, h["ns_steps"], h["eps"], torch.float64)
    rough = orthogonal(u.float(), h["ns_steps"], h["eps"], torch.float32)
    old = p.double()
    new = old - h["lr"] * (h["weight_decay"] * old + s * x)
    # 16 roundings of u, X and its sum with p, each of the size of p or of the update
    bound = 8 * h["lr"] * s * float((rough - x).norm()) + \
        16 * H * (float(old.norm()) + h["lr"] * s * 4 * float(x.norm()))
    return new, m, bound


def fill(kind, shape, rng):
    x = rng.standard_normal(shape)
    r, c = shape[-2:]
    if kind == "strong":           # a few directions and little else
        k = max(1, min(r, c) // 16)
        x = rng.standard_normal((*shape[:-1], k)) @ rng.standard_normal((*shape[:-2], k, c)) + 0.01 * x
    elif kind == "rank 1":
        x = rng.standard_normal((*shape[:-1], 1)) @ rng.standard_normal((*shape[:-2], 1, c))
    elif kind == "rows":           # gradients of a few rows only, as an embedding's
        x[..., rng.random(r) < 0.8, :] = 0
    elif kind == "large":
        x = x * 1e30
    elif kind == "tiny":
        x = x * 1e-33
    return torch.from_numpy(x.astype(np.float32))


HYPER = dict(momentum=0.95, nesterov=True, ns_steps=5, eps=1e-7, weight_decay=0.1, match_rms=None, grad_scale=1.0)


def check(shapes, kind="noise", pd=F32, gd=F32, copy=False, lr=0.02, steps=1, seed=0, **hyper):
    h = {**HYPER, **hyper, "lr": lr}
    rng = np.random.default_rng(seed)
    g = [fill(kind, s, rng).to(gd) for s in shapes]
    p = [torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.02).to(pd) for s in shapes]
    m = [fill(kind, s, rng) for s in shapes]
    on = lambda ts: [t.to(DEV) for t in ts]  # noqa: E731
    gp, gg, gm = on(p), on(g), on(m)
    copies = [torch.full(s, float("nan"), dtype=BF16, device=DEV) for s in shapes] if copy else None
    opt = ar.Muon(gp, gg, copies, state={"momentum": gm}, **{k: v for k, v in h.items() if k != "lr"})
    for _ in range(steps):
        opt.step(lr)
    for i in range(len(shapes)):
        want, bound = p[i], 0.0
        mom = m[i]
        for _ in range(steps):
            want, mom, b = expected(want.float() if pd == F32 else want, g[i], mom.float(), h)
            bound += b
            if pd == BF16:
                bound += 2.0 ** -8 * float(want.norm())
                want = want.to(BF16)
            else:
                bound += H * float(want.norm())
        got = gp[i].cpu().double()
        size = mom.abs() + g[i].double().abs()
        assert bool(((gm[i].cpu().double() - mom).abs() <= steps * 4 * H * size + 1e-44).all()), f"{shapes[i]}: momentum"
        off = float((got - want.double()).norm())
        assert off <= bound, f"{shapes[i]} {kind}: {off:.3g} of {bound:.3g}"
        if copy:
            assert torch.equal(copies[i], gp[i].to(BF16))


@pytest.mark.parametrize("shape", [
    (1, 1), (1, 50), (50, 1), (2, 3), (16, 16), (61, 100), (100, 61), (64, 64), (63, 65), (64, 512), (512, 64),
    (128, 129), (130, 127), (200, 700), (300, 300), (5, 48, 96), (3, 2, 70, 33), (1, 2048), (17, 5000),
])
@pytest.mark.parametrize("kind", ["noise", "strong"])
def test_one_tensor(shape, kind):
    announce(f"{shape} {kind}")
    check([shape], kind)


@pytest.mark.parametrize("pd,gd,copy", [(F32, F32, True), (F32, BF16, True), (F32, BF16, False), (BF16, BF16, False),
                                        (BF16, F32, False)])
def test_types_of_many_tensors(pd, gd, copy):
    announce(f"types {pd} {gd} {copy}")
    check([(100, 61), (7, 200), (4, 64, 128), (256, 64), (1, 9)], "strong", pd, gd, copy)


@pytest.mark.parametrize("shapes", [
    [(128, 64), (64, 128), (16, 16), (2, 31, 127)], [(128, 65), (65, 66), (1, 1), (128, 128)],
    [(64, 64), (33, 7), (3, 17, 48)],
])
@pytest.mark.parametrize("pd,gd,copy", [(F32, F32, True), (BF16, BF16, False)])
def test_small_matrices_together(shapes, pd, gd, copy):
    announce(f"{shapes} {pd}")
    check(shapes, "noise", pd, gd, copy)


@pytest.mark.parametrize("kind", ["rank 1", "rows", "large", "tiny"])
def test_values(kind):
    announce(kind)
    check([(96, 160), (3, 130, 70)], kind)


@pytest.mark.parametrize("hyper", [
    {"nesterov": False}, {"momentum": 0.0}, {"ns_steps": 1}, {"ns_steps": 2}, {"ns_steps": 6}, {"weight_decay": 0.0},
    {"match_rms": 0.2}, {"grad_scale": 0.125}, {"lr": 0.0}, {"eps": 1.0}, {"steps": 3},
])
def test_hyperparameters(hyper):
    announce(str(hyper))
    check([(90, 40), (64, 200)], **hyper)


def test_wide_tiles():
    """Enough work for the larger tiles, with sizes around theirs."""
    announce("wide tiles")
    check([(24, 300, 500), (130, 1000), (1000, 129), (20, 256, 256)], "strong", F32, BF16, True)


def test_zeros_and_values_that_are_not_finite():
    """They stay in their own matrix."""
    p = [torch.ones(4, 70, 90, device=DEV)]
    g = [torch.randn(4, 70, 90, device=DEV)]
    g[0][1] = 0
    g[0][2, 3, 4] = float("nan")
    g[0][3, 5, 6] = float("inf")
    alone = [p[0][:1].clone()]
    ar.Muon(alone, [g[0][:1].clone()], weight_decay=0.5).step(0.25)
    ar.Muon(p, g, weight_decay=0.5).step(0.25)
    assert torch.equal(p[0][0], alone[0][0])
    assert bool((p[0][1] == 0.875).all())          # decay alone
    assert bool(p[0][2].isnan().all() and p[0][3].isnan().all())


@pytest.mark.parametrize("shape", [(8, 8), (100, 61), (200, 300)])
def test_zeros_without_an_eps(shape):
    p, g = [torch.ones(shape, device=DEV)], [torch.zeros(shape, device=DEV)]
    ar.Muon(p, g, eps=0.0, weight_decay=0.5).step(0.25)
    assert bool((p[0] == 0.875).all())


def test_flat_gradients_and_state():
    p = [torch.randn(40, 30, device=DEV)]
    q, g, m = [p[0].clone()], torch.randn(1200, device=DEV), torch.randn(1200, device=DEV)
    ar.Muon(p, [g.view(40, 30)], state={"momentum": [m.view(40, 30).clone()]}).step(0.1)
    ar.Muon(q, [g], state={"momentum": [m]}).step(0.1)
    assert torch.equal(p[0], q[0])


def test_empty_tensors_and_odd_addresses():
    flat = torch.randn(100 * 61 + 3, device=DEV)
    p = [flat[3:].view(100, 61).clone(), torch.empty(0, 5, 6, device=DEV), torch.empty(3, 0, 6, device=DEV)]
    q = flat[3:].view(100, 61)
    g = torch.randn(100 * 61 + 1, device=DEV).bfloat16()
    ar.Muon(p, [g[1:].view(100, 61).clone(), torch.empty(0, 5, 6, device=DEV).bfloat16(),
                torch.empty(3, 0, 6, device=DEV).bfloat16()]).step(0.1)
    ar.Muon([q], [g[1:].view(100, 61)]).step(0.1)
    assert torch.equal(p[0], q)
    ar.Muon(p[1:], p[1:]).step(0.1)                # nothing to do


def test_autograd_notices_a_step():
    w = torch.randn(20, 30, device=DEV, requires_grad=True)
    loss = (w * w).sum()
    ar.Muon([w.detach()], [torch.randn(20, 30, device=DEV)]).step(0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def twins(seed=1):
    gen = torch.Generator(DEV).manual_seed(seed)
    new = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    p, g = [new(300, 200), new(3, 64, 96)], [new(300, 200), new(3, 64, 96)]
    return ar.Muon(p, g, weight_decay=0.1), ar.Muon([t.clone() for t in p], g, weight_decay=0.1)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a.params + a.state["momentum"], b.params + b.state["momentum"]))


def test_the_same_step_gives_the_same_bits():
    a, b = twins()
    for _ in range(5):
        a.step(0.02)
        b.step(0.02)
    assert same(a, b)


def test_captured_and_replayed_beside_eager_steps():
    a, b = twins()
    c, d = twins(2)
    a.step(0.02), b.step(0.02)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.step(0.02)
    for k in range(4):
        for t in a.grads:
            t.normal_()
        graph.replay()
        c.step(0.01)
        b.step(0.02)
        d.step(0.01)
        torch.cuda.synchronize()
        assert same(a, b) and same(c, d), k


def test_on_a_named_stream_with_the_object_dropped():
    p, q = torch.ones(400, 300, device=DEV), torch.ones(400, 300, device=DEV)
    g = torch.randn(400, 300, device=DEV)
    ar.Muon([q], [g]).step(0.1)
    opt = ar.Muon([p], [g])
    like = [torch.empty_like(g), torch.empty_like(opt._workspace), torch.empty_like(opt._device)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    opt.step(0.1, stream=side)
    used = {t.data_ptr() for t in (g, opt._workspace, opt._device, *opt.state["momentum"])}
    del opt, g
    again = [torch.zeros_like(t) for t in like for _ in range(3)]
    assert not used & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert torch.equal(p, q)


def test_refusals():
    m = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
    p = m(8, 8)
    bad = [
        (ValueError, lambda: ar.Muon([], [])), (TypeError, lambda: ar.Muon([p.cpu()], [p])),
        (ValueError, lambda: ar.Muon([m(8)], [m(8)])), (TypeError, lambda: ar.Muon([p.half()], [p])),
        (TypeError, lambda: ar.Muon([p], [p.half()])), (ValueError, lambda: ar.Muon([p], [m(8, 9)])),
        (ValueError, lambda: ar.Muon([p], [m(8, 8), m(8, 8)])), (ValueError, lambda: ar.Muon([p.t()[:4]], [m(4, 8)])),
        (TypeError, lambda: ar.Muon([p.bfloat16()], [m(8, 8)], [m(8, 8, dt=BF16)])),
        (TypeError, lambda: ar.Muon([p], [m(8, 8)], [m(8, 8)])),
        (ValueError, lambda: ar.Muon([p], [m(8, 8)], state={})),
        (TypeError, lambda: ar.Muon([p], [m(8, 8)], state={"momentum": [m(8, 8, dt=BF16)]})),
        (ar.ArError, lambda: ar.Muon([p], [p])),                              # a gradient in the parameter
        (ar.ArError, lambda: ar.Muon([p], [m(8, 8)], state={"momentum": [p]})),
        (ValueError, lambda: ar.Muon([p], [m(4, 16)])),                       # as many elements, another matrix
        (ValueError, lambda: ar.Muon([p], [m(8, 8)], [m(1, 8, 8, dt=BF16)])),
        (ValueError, lambda: ar.Muon([p], [m(8, 8)], state={"momentum": [m(16, 4)]})),
        (ValueError, lambda: ar.Muon([p], [m(8, 8)], ns_steps=2.5)),
        (ValueError, lambda: ar.Muon([p], [m(8, 8)], match_rms=0.0)),
    ]
    bad += [(ar.ArError, lambda k=k, v=v: ar.Muon([p], [m(8, 8)], **{k: v}).step(0.1))
            for k, v in (("ns_steps", 0), ("ns_steps", 33), ("momentum", 1.0), ("momentum", -0.1), ("eps", -1.0),
                         ("eps", float("nan")), ("weight_decay", -0.1), ("grad_scale", float("inf")))]
    bad += [(ar.ArError, lambda v=v: ar.Muon([p], [m(8, 8)]).step(v)) for v in (-1.0, float("nan"), float("inf"))]
    ar.debug_fail_launch(1)
    try:
        for i, (error, call) in enumerate(bad):
            with pytest.raises(error):
                call()
                raise AssertionError(f"case {i} was taken")
        with pytest.raises(ar.ArError, match="HIP"):
            ar.Muon([p], [m(8, 8)]).step(0.1)
    finally:
        ar.debug_fail_launch(0)
    assert not p.any()
