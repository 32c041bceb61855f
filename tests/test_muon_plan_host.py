"""CPU tests of what a Muon plan holds: how its tiles are shared out, and what
a step needs to work in.  Nothing is launched."""

import ctypes

import pytest

import tree_allreduce_algorithms_amd as ar
from test_experts_host import HIP, at, built_library, head, plan, step, tensors  # noqa: F401


def parts(image, table, count):
    """{parts of a tile: tiles that have so many} of a table of the plan."""
    small, large = head(image)
    n, seen = small[count], {}
    words = (ctypes.c_uint32 * (8 * n)).from_buffer(image, large[table])
    for i in range(n):
        if words[8 * i] != 2 ** 32 - 1:
            seen[words[8 * i], words[8 * i + 1]] = words[8 * i + 5]
    return {p: list(seen.values()).count(p) for p in set(seen.values())}


@pytest.mark.parametrize("short,long", [(2048, 2048), (2048, 4096), (2176, 2304)])
@pytest.mark.parametrize("less", [1, 63, 64, 68, 127])
def test_a_padded_side_is_shared_out_as_the_whole_one(short, long, less):
    """Tiles of 128 for X and 64 for its square: sides that are rounded up to the
    same size have the same tiles, and as many parts of them."""
    whole, padded = (plan(tensors([(1, s, long)]))[1] for s in (short, short - less))
    assert head(whole)[0]["side"] == head(padded)[0]["side"] == 128
    assert head(whole)[0]["square_side"] == head(padded)[0]["square_side"] == 64
    for table, count in (("squares_at", "squares"), ("polys_at", "polys"), ("tiles_at", "tiles")):
        assert parts(whole, table, count) == parts(padded, table, count), table


def padded(shapes, side):
    up = lambda x: -(-x // side) * side  # noqa: E731
    return sum(n * (8 * up(r) * up(c) + 8 * up(min(r, c)) ** 2) for n, r, c in shapes)


@pytest.mark.parametrize("shapes", [[(1, 1, 1)], [(3, 61, 100)], [(100_000, 8, 8)], [(7, 128, 128), (2, 1, 128)]])
def test_steps_of_small_matrices_work_in_no_memory(shapes):
    image = plan(tensors(shapes))[1]
    assert ar.lib().ar_muon_workspace_used(image) == 0
    assert step(image, workspace=at(100)) == HIP            # the device plan's own address will do


@pytest.mark.parametrize("shapes,side", [([(1, 129, 1)], 64), ([(60, 16, 4096)], 128), ([(1, 1, 4_000_000)], 128),
                                         ([(1, 300, 300), (300, 16, 16)], 128), ([(3, 1000, 700)], 64),
                                         ([(2, 500, 700)], 64), ([(1, 2100, 4000)], 128)])
def test_memory_of_other_matrices_is_what_the_header_says(shapes, side):
    image = plan(tensors(shapes))[1]
    used = ar.lib().ar_muon_workspace_used(image)
    assert used == ar.lib().ar_muon_workspace(image)
    assert head(image)[0]["side"] == side
    assert padded(shapes, side) <= used <= padded(shapes, side) + 34_000_000


def test_a_plan_that_is_none_has_no_memory():
    assert ar.lib().ar_muon_workspace_used(None) == 0
    assert ar.lib().ar_muon_workspace_used((ctypes.c_char * 4096)()) == 0
    assert ar.lib().ar_muon_workspace_used(plan(tensors([(0, 8, 8)]))[1]) == 0
