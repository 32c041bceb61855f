"""CPU tests of what a Muon plan holds: how its tiles are shared out, and what
a step needs to work in.  Nothing is launched."""

import ctypes

import pytest

from test_experts_host import BF16, F32, built_library, head, plan, tensors  # noqa: F401


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
