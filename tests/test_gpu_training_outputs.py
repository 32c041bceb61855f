"""The training calls' outputs as tensors: what a user does with them besides computing."""

import io

import torch
import pytest

import tree_allreduce_algorithms_amd as ar
from test_gpu_route import gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu


def outputs(ranks=3, tokens=50, experts=24, k=4):
    r = ar.route([torch.randn(tokens, experts, device="cuda") for _ in range(ranks)], k)
    return {"indices": r.indices, "weights": r.weights, "counts": r.counts, "share": r.share, "loss": r.loss}


def test_a_routing_can_be_saved_and_loaded():
    out = outputs()
    file = io.BytesIO()
    torch.save(out, file)
    file.seek(0)
    back = torch.load(file, weights_only=True)
    assert all(torch.equal(out[k], back[k]) and out[k].dtype == back[k].dtype for k in out)


def test_every_output_has_a_storage_of_its_own():
    out = outputs()
    assert len({t.untyped_storage().data_ptr() for t in out.values()}) == len(out)
    for t in out.values():
        assert t.storage_offset() == 0 and t.is_contiguous() and t.device == torch.device("cuda:0")
        assert t.untyped_storage().nbytes() == t.numel() * t.element_size()
        assert not t.requires_grad and t.grad_fn is None


def test_outputs_of_no_tokens_and_in_place_changes():
    out = outputs(tokens=0)
    assert out["indices"].shape == (3, 0, 4) and float(out["loss"]) == 0
    out = outputs()
    keep = out["indices"].clone()
    out["weights"].mul_(2)
    out["share"].zero_()
    assert torch.equal(out["indices"], keep) and float(out["loss"]) > 0
