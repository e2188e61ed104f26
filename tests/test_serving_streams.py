"""Which streams a framework object's tensors are marked as used on (no GPU: a
stand-in for the tensors)."""
import types

import torch

from ssm_decode_amd.layer import _StreamUses


class Tensor:
    device = types.SimpleNamespace(type="cuda", index=0)

    def __init__(self):
        self.streams = []

    def record_stream(self, st):
        self.streams.append(st)


def test_every_other_stream_is_marked_once(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7, raising=False)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: "default")
    a, b = Tensor(), Tensor()
    uses = _StreamUses(a, None, b)
    assert [uses.add(h) for h in (7, 9, 0, 9, 7, 0)] == [7, 9, 0, 9, 7, 0]
    assert a.streams == b.streams == [("external", 9), "default"]


def test_tensors_in_host_memory_need_no_marks():
    assert _StreamUses(torch.empty(3), None).add(5) == 5
