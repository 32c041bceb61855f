"""CPU test of what the training module tells autograd about tensors that a
kernel has written."""

import pytest
import torch

from tree_allreduce_algorithms_amd import training


def test_written_tensors_fail_a_backward_that_saved_them():
    w = torch.ones(4, requires_grad=True)
    flat = torch.zeros(8)
    view = flat[2:6]
    y = (w * w).sum() + (w * view).sum()
    before = [t._version for t in (w, view, flat)]
    training._training.written([w, view])
    assert [t._version for t in (w, view, flat)] == [v + 1 for v in before]     # a view's base too
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_written_takes_what_has_no_version():
    with torch.inference_mode():
        t = torch.zeros(3)
    training._training.written([t, torch.zeros(0)])
    training._training.written([])
    for bad in (None, (t,), [None]):
        with pytest.raises(TypeError):
            training._training.written(bad)
