"""Training calls in captured graphs, beside eager ones."""

import pytest
import torch

import tree_allreduce_algorithms_amd as ar
from test_gpu_adamw import F32, HYPER, gpu_ready, make  # noqa: F401

pytestmark = pytest.mark.gpu


def twins(bits):
    p, g, _, state = make([5000, 300], bits, F32, F32, False, 0, 17)
    q = [t.clone() for t in p]
    other = {k: [t.clone() for t in ts] for k, ts in state.items()}
    return (ar.AdamW(p, g, state_bits=bits, state=state, **HYPER),
            ar.AdamW(q, g, state_bits=bits, state=other, **HYPER))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("named", [False, True])
def test_steps_clipped_by_a_captured_norm(bits, named):
    """Replay and step, several times, against an object that does both eagerly."""
    a, b = twins(bits)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        norm = a.grad_norm(max_norm=0.5, stream=side if named else None)
    for k in range(5):
        for t in a.grads:
            t.normal_(0, 1 + k)
        graph.replay()
        a.step(1e-3, clip=True)
        want = b.grad_norm(max_norm=0.5)
        b.step(1e-3, clip=True)
        torch.cuda.synchronize()
        assert torch.equal(norm, want), k
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params)), k
        for key in a.state:
            assert all(torch.equal(x, y) for x, y in zip(a.state[key], b.state[key])), (k, key)
    assert a.steps == b.steps == 5


def test_a_captured_norm_that_has_not_run_shows():
    """Capture alone computes nothing: without a replay the factor is the plan's
    own, NaN, and not a 0 that would drop the gradients."""
    a, _ = twins(32)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.grad_norm(max_norm=0.5)
    a.step(1e-3, clip=True)
    assert all(torch.isnan(t).all() for t in a.params)


def test_a_captured_norm_without_a_bound_is_none_to_clip_by():
    a, _ = twins(32)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.grad_norm()
    graph.replay()
    with pytest.raises(ValueError, match="clip"):
        a.step(1e-3, clip=True)


def test_replays_of_the_router_run_beside_eager_calls():
    """Replays on one stream while eager calls run on another: each has sums of its own."""
    logits = [torch.randn(4000, 64, device="cuda") for _ in range(4)]
    dw = [torch.randn(4000, 4, device="cuda") for _ in range(4)]
    one = torch.ones((), device="cuda")

    def both():
        r = ar.route(logits, 4, renormalize=True)
        return r.indices, r.weights, r.counts, r.loss, ar.route_grad(logits, r, dw, one)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = both()
    side = torch.cuda.Stream()
    for k in range(6):
        for t in logits:
            t.normal_()
        want = both()
        torch.cuda.synchronize()
        for _ in range(10):
            with torch.cuda.stream(side):
                graph.replay()
            eager = both()
        torch.cuda.synchronize()
        for a, b, c in zip(replayed, eager, want):
            assert torch.equal(a, c) and torch.equal(b, c), k
