"""CPU test of which streams the allocator is told of."""

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
