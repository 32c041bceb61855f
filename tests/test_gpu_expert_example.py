"""The layer of experts trained on logical ranks: it runs, its gradients are those
of the formula, and what a step leaves fits together."""

import importlib.util
import os
import subprocess
import sys

import pytest
import torch

import tree_allreduce_algorithms_amd as ar
from conftest import ROOT
from test_gpu_experts import gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu

PATH = os.path.join(ROOT, "examples", "moe_muon_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_muon_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs():
    done = subprocess.run([sys.executable, PATH, "--steps", "3"], capture_output=True, text=True, timeout=100)
    assert done.returncode == 0, done.stderr[-2000:]
    assert done.stdout.count("step") == 3 and "nan" not in done.stdout


def test_gradients_are_the_formula_s(example):
    """Of the error on one rank's tokens, the router's choice held: 2-norms, with
    three roundings of half a bfloat16 step (2^-8) between the weights and the sums,
    three more on the way back, and twice that for ReLUs that a rounding turns."""
    t = example.Trainer(seed=1)
    x = [torch.randn(example.TOKENS, example.DIM, device="cuda").bfloat16() for _ in range(example.RANKS)]
    t.backward(x)
    routing = ar.route([v.float() @ t.router for v in x], example.TOP_K, renormalize=True)
    for r in (0, example.RANKS - 1):
        index, gate = routing.indices[r].long(), routing.weights[r].double()

        def sums(w1, w2):
            hidden = torch.relu((x[r].double()[:, None, :, None] * w1[index]).sum(2))
            return (gate[..., None] * (hidden[..., None] * w2[index]).sum(2)).sum(1)

        w1, w2 = (c[r].double().requires_grad_() for c in t.copies)
        target = sums(*(w.double() for w in t.teacher))
        (sums(w1, w2) - target).square().mean().backward()
        for got, want in ((t.grads[0][r], w1.grad), (t.grads[1][r], w2.grad)):
            off = float((got.double() - want).norm() / want.norm())
            assert off <= 2 * 6 * 2.0 ** -8, off


def test_a_step_leaves_the_same_weights_everywhere(example):
    t = example.Trainer(seed=2)
    for _ in range(2):
        t.step(0.05)
    for i, copies in enumerate(t.copies):
        whole = torch.cat([p for p in t.muon.params[i * example.RANKS:(i + 1) * example.RANKS]])
        for c in copies:
            assert torch.equal(c, whole.bfloat16())
