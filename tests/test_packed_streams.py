"""The stream argument of the packed operators, without a GPU: the call is
recorded in place of being made."""
import contextlib

import pytest
import torch

from compressive_memory_segment_b200 import binding as bd


class FakeStream:
    def __init__(self, handle, device=None):
        self.handle, self.device = handle, torch.device(device) if device is not None else torch.device("cuda", 0)


def test_a_stream_of_another_device_is_not_dropped(monkeypatch):
    """A raw handle belongs to the tensors' device; a stream object of another device is refused, not ignored."""
    used, calls = [], []

    @contextlib.contextmanager
    def stream(s):
        used.append(s)
        yield

    monkeypatch.setattr(bd, "_call", lambda fn, dev, *args: calls.append(args))
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(bd, "_device_of", lambda x: torch.device("cuda", 1), raising=False)
    x, off = torch.zeros(8, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 4, 8], dtype=torch.int32)
    bd.packed_forward(x, x, x, off, stream=1234)
    assert used[-1].handle == 1234 and used[-1].device == torch.device("cuda", 1)
    n = len(calls)
    with pytest.raises(ValueError):
        bd.packed_forward(x, x, x, off, stream=FakeStream(5, "cuda:0"))
    assert len(calls) == n
    bd.packed_forward(x, x, x, off, stream=FakeStream(5, "cuda:1"))
    assert len(calls) == n + 1


def test_a_stream_for_tensors_without_a_device(monkeypatch):
    x, off = torch.zeros(8, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 4, 8], dtype=torch.int32)
    for stream in (1234, FakeStream(5, "cuda:0")):
        with pytest.raises(ValueError):
            bd.packed_forward(x, x, x, off, stream=stream)
    with pytest.raises(TypeError):
        bd.packed_forward(stream=1234)
