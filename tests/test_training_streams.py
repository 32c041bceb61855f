"""CPU tests of which streams the allocator is told of, and which keep a
router's workspace."""

import torch

from tree_allreduce_algorithms_amd import training


class Tensor:
    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


class Stream:
    def __init__(self, name):
        self.name = name


class External(Stream):
    pass


def test_named_torch_streams_are_recorded_and_no_others(monkeypatch):
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    side = Stream("side")
    a, b, c = Tensor(), Tensor(), Tensor()
    for stream in (None, 12345, External("external")):
        training._in_use(stream, [a, b], None, (c,))
        assert not a.streams and not b.streams and not c.streams
    training._in_use(side, [a, b], None, (c,))
    assert a.streams == b.streams == c.streams == [side]


def test_only_streams_that_last_keep_a_workspace(monkeypatch):
    """(handle, id) of the null stream, one of torch's own, and an external one."""
    made, capturing = [], False
    real = torch.zeros

    def zeros(n, dtype, device):
        made.append(real(1))
        return made[-1]

    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(training, "_route_workspaces", {})
    for handle, stream_id, kept in ((0, 0, True), (0x7F01, 35, True), (0x7F02, 0x7F02, False)):
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: type("S", (), {"stream_id": stream_id}))
        first, second = (training._route_workspace(0, handle) for _ in range(2))
        assert (first is second) == kept
        assert ((0, handle) in training._route_workspaces) == kept
    assert len(made) == 4
    capturing = True
    assert training._route_workspace(0, 0x7F01) is not training._route_workspaces[0, 0x7F01]
    assert training._route_workspace(0, 0) is training._route_workspaces[0, 0]


def test_an_optimizer_records_a_torch_stream_once_also_after_its_raw_handle(monkeypatch):
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    opt = training.AdamW.__new__(training.AdamW)
    opt.params, opt.grads, opt.copies, opt.state = [Tensor()], [Tensor()], None, {"exp_avg": [Tensor()]}
    opt._device, opt._norm, opt._streams = Tensor(), Tensor(), set()
    tensors = [*opt.params, *opt.grads, *opt.state["exp_avg"], opt._device, opt._norm]
    opt._on(77, 77)
    assert not any(t.streams for t in tensors)
    side = Stream("side")
    for _ in range(3):
        opt._on(side, 77)
    assert all(t.streams == [side] for t in tensors)
