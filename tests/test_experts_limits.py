"""CPU tests of how much the experts' calls take.  Nothing is launched: an armed
injection stands in for the launch."""

import pytest

from test_experts_host import HIP, UNSUPPORTED, built_library, combine, combine_grad  # noqa: F401


@pytest.mark.parametrize("top_k,want", [(2 ** 31 - 4, HIP), (2 ** 31 - 3, UNSUPPORTED), (2 ** 31 - 1, UNSUPPORTED)])
def test_sums_refuse_more_choices_than_their_counter_reaches(top_k, want):
    assert combine(tokens=1, top_k=top_k) == want
    assert combine_grad(tokens=1, top_k=top_k) == HIP          # which counts pairs, in 32 bits without a sign
