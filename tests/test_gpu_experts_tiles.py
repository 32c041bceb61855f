"""The experts' products in each of their tiles, on the GPU, against the
definition in 64 bits (tolerances are those of test_gpu_experts).

Which kernel a product runs in goes by its rows an expert and its sizes, so the
wide tiles, and the stores past the caches, need thousands of rows.  Here each
case says which it is meant for; `tiles_of` repeats the rule, so that a case
does not leave its kernel unnoticed.
"""

import sys

import numpy as np
import pytest
import torch

import tree_allreduce_algorithms_amd as ar
import test_gpu_experts as plain
from test_gpu_experts import BF16, F32, bf16, choices, gpu_ready, grouped, near, order_of  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
PAST = 32 << 20               # results of so many bytes are stored past the caches


def announce(msg):
    print(f"[gpu-tiles] {msg}", file=sys.__stderr__, flush=True)


def tiles_of(pairs, experts, n_out, turned, direct):
    each = pairs // min(pairs, experts)
    if each <= 16:
        return "16 x 64"
    if each <= (64 if direct else 128) or (n_out <= 128 and direct) or pairs // 128 * -(-n_out // 256) < 256:
        return "64 x 128"
    if not direct:
        return "128 x 128"
    return "256 x 256" if each >= 1024 and turned else "128 x 256"


@pytest.mark.parametrize("tokens,k,experts,n_in,n_out,turned,kind,tile,past", [
    # sizes off the tiles and steps, uneven rows, padded batches; steps of one, two, three and more
    (8200, 2, 40, 136, 776, False, "skewed", "128 x 256", False),
    (8200, 2, 40, 136, 776, True, "skewed", "128 x 256", False),
    (8200, 2, 100, 24, 776, False, "masked", "128 x 256", False),
    (8200, 2, 100, 40, 776, True, "masked", "128 x 256", False),
    (11000, 3, 1, 72, 520, False, "masked", "128 x 256", False),       # one expert
    (16500, 1, 250, 520, 520, True, "even", "128 x 256", False),       # 66 rows an expert
    (8200, 2, 40, 96, 1024, False, "even", "128 x 256", True),
    (8200, 2, 40, 264, 1024, True, "even", "128 x 256", True),
    (8200, 2, 40, 2056, 1032, False, "skewed", "128 x 256", False),
    (6000, 2, 8, 200, 1032, True, "skewed", "256 x 256", False),
    (6000, 2, 8, 8, 1032, True, "masked", "256 x 256", False),
    (4100, 8, 32, 1032, 264, True, "masked", "256 x 256", False),
    (6000, 2, 8, 136, 1408, True, "one", "256 x 256", True),
    (6000, 2, 3, 72, 1408, True, "masked", "256 x 256", True),
    # not in 16-byte pieces
    (8200, 2, 40, 135, 777, False, "skewed", "128 x 128", False),
    (8200, 2, 40, 135, 777, True, "skewed", "128 x 128", False),
    (8200, 2, 40, 3, 776, False, "masked", "128 x 128", False),
    (8200, 2, 40, 67, 1024, False, "masked", "128 x 128", True),
    (8200, 2, 40, 67, 1024, True, "masked", "128 x 128", True),
    # few rows an expert, many results
    (8200, 4, 1000, 72, 512, False, "even", "64 x 128", True),
    (8200, 4, 1000, 72, 512, True, "even", "64 x 128", True),
    (8200, 4, 1000, 33, 512, False, "even", "64 x 128", True),
    (8200, 4, 1000, 33, 512, True, "even", "64 x 128", True),
    # all rows to a few of many experts: the tiles are chosen as if they were even
    (2000, 2, 256, 520, 776, False, "one", "16 x 64", False),
    (2000, 2, 256, 520, 776, True, "one", "16 x 64", False),
])
def test_matmul_in(tokens, k, experts, n_in, n_out, turned, kind, tile, past):
    announce(f"matmul {tokens} {k} {experts} {n_in} {n_out} turned={turned} {kind} {tile} past={past}")
    direct = n_in % 8 == 0 and n_out % 8 == 0
    assert tiles_of(tokens * k, experts, n_out, turned, direct) == tile
    assert (tokens * k * n_out * 2 >= PAST and n_out % 64 == 0) == past
    gen = np.random.default_rng(n_in * 41 + n_out)
    idx = choices(tokens, k, experts, kind, 15)
    order, _, offsets = order_of(idx, experts)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), experts)
    w = bf16(gen, experts, n_out, n_in).transpose(1, 2) if turned else bf16(gen, experts, n_in, n_out)
    for gather in (True, False):
        x = bf16(gen, tokens if gather else tokens * k, n_in)
        y = ar.expert_matmul(x, w, o, gather=gather)
        want, size = grouped(x, w, order, offsets, k, gather)
        near(y, want, size, n_in, f"y gather={gather}")
        assert not y[int(offsets[-1]):].any()


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("experts,n_out", [(40, 776), (8, 1032)])
def test_wide_tiles_of_views(experts, n_out, turned):
    """Rows and matrices cut out of larger tensors that hold NaN around them."""
    announce(f"views {experts} {n_out} turned={turned}")
    gen = np.random.default_rng(17)
    tokens, k, n_in = 8200, 2, 136
    idx = choices(tokens, k, experts, "masked", 16)
    order, _, offsets = order_of(idx, experts)
    o = ar.expert_order(torch.from_numpy(idx).to(DEV), experts)
    x = torch.full((tokens + 1, n_in + 24), float("nan"), dtype=BF16, device=DEV)[:tokens, 8:8 + n_in]
    x.copy_(bf16(gen, tokens, n_in))
    big = torch.full((experts, n_in + 16, n_out + 16), float("nan"), dtype=BF16, device=DEV)
    if turned:
        big = big.transpose(1, 2).contiguous().transpose(1, 2)
    w = big[:, 8:8 + n_in, 8:8 + n_out].copy_(bf16(gen, experts, n_in, n_out))
    want, size = grouped(x, w, order, offsets, k, True)
    near(ar.expert_matmul(x, w, o, gather=True), want, size, n_in, "y")


@pytest.mark.parametrize("tokens,k,experts,n_in,n_out,kind,dtype", [
    # stored past the caches: two steps under way, one, and sizes not in 16-byte pieces
    (1500, 2, 64, 512, 256, "skewed", F32), (1500, 2, 64, 512, 512, "masked", BF16),
    (700, 2, 8, 1024, 1024, "masked", F32), (900, 1, 16, 1000, 1088, "skewed", BF16),
    (700, 2, 8, 1025, 1024, "masked", F32), (600, 2, 40, 705, 640, "skewed", BF16),
    # tiles that the XCDs do not share evenly, of an odd number of experts
    (3000, 2, 33, 136, 1288, "skewed", F32), (3000, 2, 7, 392, 776, "masked", F32),
])
def test_weight_grad_in(tokens, k, experts, n_in, n_out, kind, dtype):
    for gather in (True, False):
        plain.test_weight_grad(tokens, k, experts, n_in, n_out, kind, gather, dtype)


@pytest.mark.parametrize("tokens,k,experts,size,kind", [
    (4200, 4, 8, 1024, "masked"),       # sums past the caches, of more than two choices
    (16800, 4, 8, 1001, "masked"),      # the gradient's reads past them, rows not in 16-byte pieces
    (16800, 4, 8, 1000, "skewed"),      # and rows that are not whole lines
])
def test_sums_in(tokens, k, experts, size, kind):
    plain.test_combine_and_its_gradient(tokens, k, experts, size, kind)
