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
