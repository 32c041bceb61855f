"""AdamW over arrays that begin off the 16-byte grid."""

import pytest
import torch

import tree_allreduce_algorithms_amd as ar
from test_gpu_adamw import F32, BF16, HYPER, announce, check_step, gpu_ready, make  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = ["f32 f32", "f32 bf16", "f32 f32 copy", "f32 bf16 copy", "bf16 f32", "bf16 bf16"]


def kinds_of(kind):
    dt = {"f32": F32, "bf16": BF16}
    return [dt[k] for k in kind.split()[:2]] + [kind.endswith("copy")]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("offset", [2, 4, 12])
@pytest.mark.parametrize("bits", [32, 8])
def test_arrays_at_any_element(bits, offset, kind):
    """A bfloat16 array 4 elements past a 16-byte boundary takes the wide path,
    8 bytes off; 2 elements past, the one for any alignment."""
    announce(f"offset {bits} {offset} {kind}")
    pd, gd, copy = kinds_of(kind)
    p, g, copies, state = make([4096, 1024 * 3 + 17, 9000], bits, pd, gd, copy, offset, 13)
    opt = ar.AdamW(p, g, copies, state_bits=bits, state=state, steps=4, **HYPER)
    for max_norm in (1.0, None):
        check_step(opt, bits, 1e-3, max_norm)


def parts_of(tensors, cuts):
    return [[t[a:b] for t in tensors] for a, b in zip(cuts, cuts[1:])]


@pytest.mark.parametrize("kind", KINDS)
def test_a_step_past_the_caches_is_that_through_them(kind):
    """One plan that reads more than 320 MiB against three that read less each
    (the accesses differ, the arithmetic does not), with a tail of odd size."""
    announce(f"past the caches {kind}")
    pd, gd, copy = kinds_of(kind)
    n, gen = 30_000_017, torch.Generator(device="cuda").manual_seed(3)
    cuts = [0, 2500 * 4096, 5000 * 4096, n]

    def fresh():
        gen.manual_seed(3)
        normal = lambda std: torch.randn(n, generator=gen, device="cuda") * std  # noqa: E731
        return (normal(0.02).to(pd), normal(1e-3).to(gd), normal(3e-4), normal(1e-3).square(),
                torch.zeros(n, device="cuda", dtype=BF16))

    p, g, m, v, c = fresh()
    assert n * (p.element_size() + g.element_size() + 8) > 320 << 20
    one = ar.AdamW([p], [g], [c] if copy else None, state={"exp_avg": [m], "exp_avg_sq": [v]}, steps=7, **HYPER)
    q, h, s, t, d = fresh()
    many = [ar.AdamW([a], [b], [e] if copy else None, state={"exp_avg": [x], "exp_avg_sq": [y]}, steps=7, **HYPER)
            for a, b, x, y, e in parts_of((q, h, s, t, d), cuts)]
    for _ in range(2):
        one.step(1e-3)
        for opt in many:
            opt.step(1e-3)
    torch.cuda.synchronize()
    assert torch.equal(g, h) and not torch.equal(p, fresh()[0])
    assert torch.equal(p, q) and torch.equal(m, s) and torch.equal(v, t) and torch.equal(c, d)


def test_offsets_past_32_bits_of_a_step_with_32_bit_states():
    """One tensor of 2^32 + 1,000 elements: its end is computed as its start is."""
    n, tail = (1 << 32) + 1000, 5000
    p, g = (torch.zeros(n, dtype=BF16, device="cuda") for _ in range(2))
    p[-tail:].normal_(0, 0.02)
    g[-tail:].normal_(0, 1)
    begin = (n - tail) // 4096 * 4096
    q, h = p[begin:].clone(), g[begin:].clone()
    big, small = ar.AdamW([p], [g], **HYPER), ar.AdamW([q], [h], **HYPER)
    for opt in (big, small):
        opt.step(1e-3)
    assert torch.equal(p[begin:], q) and not p[:10_000].any()
    for key in ("exp_avg", "exp_avg_sq"):
        assert torch.equal(big.state[key][0][begin:], small.state[key][0]) and small.state[key][0].any()
        assert not big.state[key][0][:10_000].any()
