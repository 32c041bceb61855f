"""What a Muon object of small matrices keeps on the GPU, and that its steps are
right without more."""

import pytest
import torch

import tree_allreduce_algorithms_amd as ar
from test_gpu_muon import H, HYPER, expected, gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count,rows,cols", [(100_000, 8, 8), (4096, 128, 128), (50_000, 3, 3), (2000, 100, 7)])
def test_many_small_matrices_keep_their_momentum_and_a_plan(count, rows, cols):
    gen = torch.Generator("cuda").manual_seed(rows)
    p = torch.randn(count, rows, cols, device="cuda", generator=gen)
    g = torch.randn(count, rows, cols, device="cuda", generator=gen)
    few = torch.tensor([0, 1, count // 2, count - 1])
    old, grad = p[few].cpu(), g[few].cpu()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    opt = ar.Muon([p], [g])
    kept = torch.cuda.memory_allocated() - before
    assert kept <= 4 * p.numel() + 320 * count + (1 << 20), f"{kept:,} bytes"
    opt.step(0.02)
    h = {**HYPER, "lr": 0.02, "weight_decay": 0.0}
    for i in range(len(few)):
        want, _, bound = expected(old[i], grad[i], torch.zeros(rows, cols), h)
        off = float((p[few[i]].cpu().double() - want).norm())
        assert off <= bound + H * float(want.norm()), (int(few[i]), off, bound)
