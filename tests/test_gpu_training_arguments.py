"""What the training calls refuse and take, beyond the first checks."""

import numpy as np
import pytest
import torch

import tree_allreduce_algorithms_amd as ar
from test_gpu_route import gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu


def test_route_grad_checks_the_routing_it_is_given():
    """A Routing's tensors can be replaced; none that the kernel would misread is taken."""
    x = [torch.randn(40, 16, device="cuda") for _ in range(2)]
    one = torch.ones((), device="cuda")
    want = ar.route_grad(x, ar.route(x, 3), dloss=one)
    bad = [("share", lambda t: t.bfloat16(), TypeError), ("share", lambda t: t.to(torch.uint8), TypeError),
           ("share", lambda t: t.double(), TypeError), ("share", lambda t: t[:8], ValueError),
           ("share", lambda t: torch.stack([t, t], 1)[:, 0], ValueError), ("share", lambda t: t.cpu(), TypeError),
           ("indices", lambda t: t.long(), TypeError), ("indices", lambda t: t.to(torch.int8), TypeError),
           ("indices", lambda t: t.float(), TypeError), ("indices", lambda t: t[:1], ValueError),
           ("indices", lambda t: t[:, :39], ValueError), ("indices", lambda t: t.flatten(), ValueError),
           ("indices", lambda t: t[..., :2], ValueError), ("indices", lambda t: t[..., :0], ValueError),
           ("indices", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), ValueError),
           ("indices", lambda t: torch.cat([t, t, t], -1), ValueError)]
    for i, (name, change, error) in enumerate(bad):
        r = ar.route(x, 3)
        setattr(r, name, change(getattr(r, name)))
        with pytest.raises(error):
            ar.route_grad(x, r, dloss=one)
            raise AssertionError(f"case {i} was taken")
    assert torch.equal(ar.route_grad(x, ar.route(x, 3), dloss=one), want)


def test_a_renormalize_without_a_truth_value():
    """The object's own error, before anything is enqueued."""
    x = [torch.randn(4, 16, device="cuda")]
    r = ar.route(x, 2)
    r._renormalize = np.zeros(2)
    for call in (lambda: ar.route(x, 2, renormalize=np.zeros(2)), lambda: ar.route_grad(x, r)):
        ar.debug_fail_launch(1)
        try:
            with pytest.raises(ValueError, match="truth value"):
                call()
        finally:
            ar.debug_fail_launch(0)


def test_strides_that_say_nothing_may_differ():
    """Single tokens cut out of matrices of several widths, and one expert."""
    wide = [torch.randn(5, n, device="cuda") for n in (16, 24, 40)]
    x = [t[2:3, :16] for t in wide]
    a, b = ar.route(x, 4), ar.route([t.clone() for t in x], 4)
    one = torch.ones((), device="cuda")
    assert torch.equal(a.indices, b.indices) and torch.equal(a.weights, b.weights) and torch.equal(a.loss, b.loss)
    assert torch.equal(ar.route_grad(x, a, dloss=one), ar.route_grad([t.clone() for t in x], b, dloss=one))
    empty = [t[:0, :16] for t in wide]
    assert ar.route(empty, 4).indices.shape == (3, 0, 4)
    single = [torch.randn(6, 1, device="cuda"), torch.randn(1, 6, device="cuda").t()]
    assert not ar.route(single, 1).indices.any()
    for bad in ([t[:, :16] for t in wide], [wide[0][:1], wide[0].t()[:1, :1].expand(1, 16)]):
        with pytest.raises(ValueError):
            ar.route(bad, 4)


def test_a_step_shows_in_a_backward_pass_that_saved_the_parameter():
    w = torch.ones(1000, device="cuda", requires_grad=True)
    copy = torch.zeros(1000, device="cuda", dtype=torch.bfloat16)
    opt = ar.AdamW([w], [torch.ones(1000, device="cuda")], [copy])
    y = (w * w).sum()
    versions = w._version, copy._version
    opt.grad_norm(max_norm=1.0)
    assert (w._version, copy._version) == versions
    with pytest.raises(ar.ArError):
        opt.step(-1.0)
    assert (w._version, copy._version) == versions
    opt.step(1e-3, clip=True)
    assert w._version > versions[0] and copy._version > versions[1]
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    (w * w).sum().backward()
    assert torch.equal(w.grad, 2 * w.detach())


def test_a_graphs_logits_take_the_gradient_by_hand():
    """Autograd records nothing of the router; its gradient is handed on."""
    w = torch.randn(32, 16, device="cuda", requires_grad=True)
    x = [torch.randn(50, 32, device="cuda") for _ in range(2)]
    logits = [t @ w for t in x]
    r = ar.route(logits, 2)
    assert r.weights.grad_fn is None and r.loss.grad_fn is None
    dx = ar.route_grad(logits, r, dloss=torch.ones((), device="cuda"))
    torch.autograd.backward(logits, list(dx))
    want = sum(t.double().t() @ d.double() for t, d in zip(x, dx))
    # 100 products a sum, each rounded, in any order
    bound = 101 * 2.0 ** -24 * sum(t.double().abs().t() @ d.double().abs() for t, d in zip(x, dx))
    assert ((w.grad.double() - want).abs() <= bound).all()
