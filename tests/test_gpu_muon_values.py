"""Muon's hyperparameters at the ends of their ranges, on the GPU."""

import pytest
import torch

import tree_allreduce_algorithms_amd as ar
from test_gpu_muon import H, HYPER, expected, gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(8, 8), (100, 61), (300, 200)])
def test_a_match_rms_below_float32_moves_nothing(shape):
    """It is not "none": an update of 1e-50 times a few is 0 beside any weight."""
    gen = torch.Generator("cuda").manual_seed(5)
    p = torch.randn(shape, device="cuda", generator=gen)
    old, g = p.clone(), torch.randn(shape, device="cuda", generator=gen)
    ar.Muon([p], [g], match_rms=1e-50).step(0.02)
    assert torch.equal(p, old)
    ar.Muon([p], [g], match_rms=1e-50, weight_decay=0.5).step(0.5)
    assert torch.equal(p, old * 0.75)


@pytest.mark.parametrize("shape", [(64, 96), (100, 30), (700, 200)])
def test_match_rms_is_the_same_for_either_layout(shape):
    """The update of [in, out] is that of [out, in], turned: each is within its
    bound of the formula, whose two results are the same."""
    gen = torch.Generator("cuda").manual_seed(6)
    p = torch.randn(shape, device="cuda", generator=gen)
    g = torch.randn(shape, device="cuda", generator=gen)
    q, gq = p.t().contiguous(), g.t().contiguous()
    h = {**HYPER, "lr": 0.02, "match_rms": 0.2}
    results = []
    for w, grad in ((p, g), (q, gq)):
        want, _, bound = expected(w.cpu(), grad.cpu(), torch.zeros(w.shape), h)
        ar.Muon([w], [grad], weight_decay=h["weight_decay"], match_rms=0.2).step(0.02)
        bound += H * float(want.norm())
        assert float((w.cpu().double() - want).norm()) <= bound
        results.append((want, bound))
    (a, bound), (b, other) = results
    assert float((p - q.t()).double().norm()) <= bound + other
    assert float((a - b.t()).norm()) <= 1e-10 * float(a.norm())      # products of float64 in another order
