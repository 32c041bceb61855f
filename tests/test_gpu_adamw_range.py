"""The AdamW step at the ends of the number range, against the formulas in 64
bits: gradients whose squares float32 cannot hold, and an eps that hides
nothing."""

import numpy as np
import pytest
import torch

import tree_allreduce_algorithms_amd as ar
from test_gpu_adamw import F32, BF16, HYPER, announce, check_step, gpu_ready, up  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gd", [F32, BF16])
@pytest.mark.parametrize("size", [256 * 5, 256 * 9 + 100])
def test_states_in_8_bits_hold_squares_beyond_float32(size, gd):
    """v' from 1e36 to 1e73 beside ordinary blocks: every code is the nearest
    one and the update is that of the definition."""
    announce(f"huge v {size} {gd}")
    rng = np.random.default_rng(6)
    x = rng.normal(0, 1, size)
    x[256:512] *= 1e25
    x[300] = 1e30
    x[512:768] = rng.choice([-1, 1], 256) * 10.0 ** rng.uniform(17, 38, 256)
    x[1024:1280] *= 3e21
    x[1100:1105] = 0
    x[-40:] = rng.normal(0, 1e36, 40)
    p = rng.normal(0, 0.02, size)
    opt = ar.AdamW([up(p, F32)], [up(x, gd)], state_bits=8, **HYPER)
    for _ in range(3):
        check_step(opt, 8, 1e-3, None)
    codes, scales = opt.state["exp_avg_sq"][0], opt.state["exp_avg_sq_scale"][0]
    with np.errstate(over="ignore"):
        u, r = codes.double().cpu().numpy(), scales.double().cpu().numpy().repeat(256)[:size]
        want = ((u * u * r) ** 2).astype(np.float32)
    assert np.array_equal(ar.dequantize(codes, scales).cpu().numpy(), want)


def test_what_an_element_gets_does_not_depend_on_its_block():
    """The same element beside others within and beyond float32's squares, and
    beside an infinity."""
    p = torch.full((1024,), 0.5, device="cuda")
    g = torch.linspace(-1, 1, 1024, device="cuda")
    far = g.clone()
    far[100], far[300], far[700] = 1e30, float("inf"), 1e-30
    q = p.clone()
    for x, y in ((p, g), (q, far)):
        ar.AdamW([x], [y], state_bits=8, **HYPER).step(1e-3)
    keep = far == g
    assert torch.equal(p[keep], q[keep]) and int(keep.sum()) == 1021


def update64(p, m, v, x, lr, t, betas, eps, weight_decay):
    """p' and the update u of the definition, from m, v and the scaled gradient."""
    m1 = betas[0] * m + (1 - betas[0]) * x
    v1 = betas[1] * v + (1 - betas[1]) * x * x
    u = (m1 / (1 - betas[0] ** t)) / (np.sqrt(v1 / (1 - betas[1] ** t)) + eps)
    return p - lr * (weight_decay * p + u), u


@pytest.mark.parametrize("kind", ["f32 f32", "f32 bf16 copy", "bf16 f32", "bf16 bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-20, 1e-15, 3e-12, 2e-10, 1e-8])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
def test_small_eps(bits, offset, eps, kind):
    """Gradients from 1e-30 to 1: what v' is beside them is never taken as 0."""
    announce(f"small eps {bits} {offset} {eps} {kind}")
    dt = {"f32": F32, "bf16": BF16}
    pd, gd = (dt[k] for k in kind.split()[:2])
    rng = np.random.default_rng(12)
    n = 256 * 8 + 77
    # an order of magnitude for each block of 256
    x = rng.choice([-1, 1], n) * rng.uniform(0.5, 1, n) * (10.0 ** -np.arange(0, 36, 4)).repeat(256)[:n]
    g = up(x, gd, offset)
    p = up(rng.normal(0, 0.02, n), pd, offset)
    copies = [up(np.zeros(n), BF16, offset)] if kind.endswith("copy") else None
    opt = ar.AdamW([p], [g], copies, state_bits=bits, betas=(0.9, 0.999), eps=eps, weight_decay=0.1)
    x, before = g.double().cpu().numpy(), p.double().cpu().numpy()
    opt.step(1e-3)
    want, u = update64(before, 0.0, 0.0, x, 1e-3, 1, (0.9, 0.999), eps, 0.1)
    got = p.double().cpu().numpy()
    # float32: betas (2 roundings each), m', v', root, sum, quotient, lr, and p' itself
    err = 16 * 2.0 ** -24 * (1e-3 * (np.abs(u) + 0.1 * np.abs(before))) + 2.0 ** -24 * np.abs(want)
    if eps > 4e-12:      # a subnormal v' of float32 is off by 2^-149, its root taken as 0 below 2^-126
        lost = np.sqrt(2.0 ** -126 / (1 - 0.999))
        err = err + 1e-3 * np.abs(u) * lost / (np.abs(x) + eps)
    if pd == BF16:
        err = err + 2.0 ** -8 * (np.abs(want) + err)
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= err), np.max(np.abs(got - want) / err)
    if copies:
        assert torch.equal(copies[0], p.to(BF16))


def test_a_large_eps():
    """One whose float32 reciprocal is not a normal number."""
    p = torch.zeros(3000, device="cuda")
    g = torch.full((3000,), 1e38, device="cuda")
    for bits in (32, 8):
        p.zero_()
        ar.AdamW([p], [g], state_bits=bits, betas=(0.9, 0.999), eps=1e39, weight_decay=0.0).step(1.0)
        want = -1e38 / (1e38 + 1e39)
        assert (p.double() - want).abs().max() <= 16 * 2.0 ** -24 * abs(want)
