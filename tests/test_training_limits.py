"""CPU tests of the training calls' limits: how much a plan and a decoding
take.  Nothing is launched: an armed injection stands in for the launch."""

import ctypes

import pytest

import tree_allreduce_algorithms_amd as ar
from test_training_host import A, F32, HIP, OK, UNSUPPORTED, built_library, plan, tensors, tiles_of  # noqa: F401
from tree_allreduce_algorithms_amd.binding import AdamwTensor

TILES = (1 << 22) - 1            # of 4,096 elements


@pytest.mark.parametrize("counts, want", [([TILES * 4096], OK), ([TILES * 4096 + 1], UNSUPPORTED),
                                          ([(TILES - 3) * 4096, 1, 5000], OK),
                                          ([(TILES - 2) * 4096, 1, 5000], UNSUPPORTED)])
def test_a_plan_takes_as_many_tiles_as_the_header_says(counts, want):
    status, image = plan(tensors(counts))
    assert status == want
    if want == OK:
        assert len(tiles_of(image)[2]) == TILES
    text = open(__file__.rsplit("/", 2)[0] + "/include/ar.h").read()
    assert "2^22 - 1 tiles of (up to) 4,096 elements" in text


def test_what_a_plan_refuses_has_no_size():
    table = (AdamwTensor * 1)(*tensors([TILES * 4096 + 1]))
    assert ar.lib().ar_adamw_plan_bytes(table, 1, F32, F32, 32) == 0
    room = ctypes.create_string_buffer(16)
    assert ar.lib().ar_adamw_plan(table, 1, F32, F32, 32, room, 16) == UNSUPPORTED


def test_a_decoding_takes_what_memory_can_hold():
    most = 4096 * ((1 << 24) - 1)
    f = ar.lib().ar_adamw_dequantize
    far = 1 << 42
    ar.debug_fail_launch(1)
    assert f(A, A + far, most, 1, A + 2 * far, None) == HIP            # the injected failure
    ar.debug_fail_launch(1)
    try:
        assert f(A, A + far, most + 1, 1, A + 2 * far, None) == UNSUPPORTED
    finally:
        ar.debug_fail_launch(0)
