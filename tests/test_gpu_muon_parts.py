"""The Muon step where its tiles come in parts, in 64 or 128 columns or both, on
the GPU: the sums that several blocks leave in memory and the last one joins.

The formula, and how far the result may be from it, are those of test_gpu_muon;
two steps in a row need the joins' counters to be 0 again.  Each case says
which parts it is meant to have, and its plan is asked.
"""

import sys

import pytest

import tree_allreduce_algorithms_amd as ar
from test_experts_host import head
from test_gpu_muon import BF16, F32, check, gpu_ready  # noqa: F401
from test_muon_plan_host import parts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shapes,kinds,sides,split", [
    # all three products in parts, X in 128 and its square in 64 columns
    ([(2048, 2048)], (F32, F32, False), (128, 64), {"squares": 2, "polys": 2, "tiles": 2}),
    # the same padded, and taller than wide, with another number of parts each
    ([(1980, 2048)], (F32, BF16, True), (128, 64), {"squares": 2, "polys": 2, "tiles": 2}),
    ([(4000, 2100)], (F32, F32, True), (128, 64), {"squares": 4, "polys": 2, "tiles": 2}),
    # all three in 128 columns, some of the tiles whole
    ([(2, 2850, 2900)], (BF16, BF16, False), (128, 128), {"squares": 2, "polys": 2, "tiles": 2}),
    # every tile of X X^T in parts, and those of one matrix beside whole ones
    ([(8, 250, 4096), (2, 4096, 500)], (F32, F32, False), (128, 64), {"squares": 3}),
    ([(50, 16384), (2, 2048, 2048)], (F32, BF16, False), (128, 128), {"squares": 8}),
    # few tiles, all in 64 columns
    ([(64, 5000), (100, 3000)], (F32, F32, True), (64, 64), {"squares": 4}),
])
def test_tiles_in_parts(shapes, kinds, sides, split, monkeypatch):
    print(f"[gpu-muon] parts {shapes}", file=sys.__stderr__, flush=True)
    made = []
    init = ar.Muon.__init__

    def remember(self, *a, **k):
        init(self, *a, **k)
        made.append(self)

    monkeypatch.setattr(ar.Muon, "__init__", remember)
    check(shapes, "strong", *kinds, ns_steps=2, steps=2)
    image = made[0]._host
    small = head(image)[0]
    assert (small["side"], small["square_side"]) == sides
    found = {t: parts(image, f"{t}_at", t) for t in ("squares", "polys", "tiles")}
    for table, most in split.items():
        assert max(found[table]) == most, found
