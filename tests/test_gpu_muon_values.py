"""Muon's hyperparameters at the ends of their ranges, on the GPU."""

import pytest
import torch

import tree_allreduce_algorithms_amd as ar
from test_gpu_muon import gpu_ready  # noqa: F401

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
