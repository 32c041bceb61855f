"""The example's training step: the operators and the collectives together."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    spec = importlib.util.spec_from_file_location("moe_train_step",
                                                  os.path.join(ROOT, "examples", "moe_train_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("state_bits", [32, 8])
def test_the_error_falls_and_the_copies_agree(example, state_bits):
    trainer = example.Trainer(state_bits)
    first = [float(trainer.step(1e-2)[0]) for _ in range(3)]
    for _ in range(100):
        error, balance, norm = trainer.step(1e-2)
    assert float(error) < 0.7 * max(first)
    assert 0.9 < float(balance) < example.EXPERTS and float(norm) > 0
    # every rank holds the same copies, which are the shards' weights rounded
    assert all(torch.equal(c, trainer.copies[0]) for c in trainer.copies)
    assert torch.equal(trainer.copies[0], torch.cat(trainer.optimizer.params).bfloat16())


def test_the_step_is_that_of_autograd(example):
    """The router's and the experts' gradients of one step against torch's own."""
    trainer = example.Trainer(32, seed=3)
    start = [c.clone() for c in trainer.copies]
    torch.manual_seed(11)
    trainer.step(1e-3)
    torch.manual_seed(11)
    x = [torch.randn(example.TOKENS, example.DIM, device="cuda") for _ in range(example.RANKS)]
    flat = start[0].double().cpu().requires_grad_()
    router, experts = example.split(flat)
    teacher_router, teacher_experts = example.split(trainer.teacher.double().cpu())
    total, probabilities, counts = 0.0, 0.0, torch.zeros(example.EXPERTS, dtype=torch.float64)
    for t in x:
        t = t.double().cpu()

        def mix(router, experts):
            p = torch.softmax(t @ router, -1)
            w, index = p.topk(example.TOP_K, -1)
            w = w / w.sum(-1, keepdim=True)
            return (w[:, :, None] * torch.einsum("td,tkde->tke", t, experts[index])).sum(1), p, index

        y, p, index = mix(router, experts)
        target = mix(teacher_router, teacher_experts)[0]
        total = total + (y - target).square().mean()
        probabilities = probabilities + p.sum(0)
        counts += torch.bincount(index.flatten(), minlength=example.EXPERTS).double()
    n = example.RANKS * example.TOKENS
    balance = example.EXPERTS / (example.TOP_K * n ** 2) * (counts * probabilities).sum()
    # every rank adds its own error's gradient, and all of them the balance loss's
    (total + example.BALANCE * balance).backward()
    count = trainer.count // example.RANKS
    got = torch.cat([trainer.grads[r][r * count:(r + 1) * count] for r in range(example.RANKS)])
    want = flat.grad
    # float32 sums over 512 products of a few units: 1e-5 of the largest is 80 roundings
    assert float((got.cpu().double() - want).abs().max()) <= 1e-5 * float(want.abs().max())
