"""The AdamW step at the ends of the number range, against the formulas in 64
bits: gradients whose squares float32 cannot hold."""

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
