"""Tensors that belong to one call alone, on a stream that is given as a handle, are
marked as used there, so that a temporary may be dropped behind the call (no GPU: the
calls are stopped in front of the library)."""
import types

import pytest
import torch

from ssm_decode_amd import abi, layer, serving
from ssm_decode_amd.layer import DecodeLayer
from ssm_decode_amd.serving import BeamSearch, ShortConv

from .test_sequence_abi import _Layer, lib  # noqa: F401  (lib: the library is built)

HERE = 7                                         # the current stream's handle


@pytest.fixture
def marks(monkeypatch):
    """(data pointer, stream) of every mark; tensors count as the device's."""
    seen = []
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: HERE, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: "default")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, st: seen.append((t.data_ptr(), st)))
    for name in ("sketchssm_conv", "sketchssm_beam_select", "sketchssm_reorder"):
        monkeypatch.setattr(abi, name, lambda *a: 0)
    return seen


def on(marks, tensors, stream):
    return all((t.data_ptr(), stream) in marks for t in tensors)


@pytest.mark.parametrize("handle,name", [(9, ("external", 9)), (0, "default")])
def test_tensors_of_one_call(marks, handle, name):
    i = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    lay = _Layer()
    conv = ShortConv(lay, torch.zeros(256, 4))
    t = dict(x=torch.zeros(5, 256), q=torch.zeros(5, 4, 16), k=torch.zeros(5, 4, 16), v=torch.zeros(5, 4, 32),
             seq_start=i(0, 2, 5), seqs=i(1, 0), has_state=i(1, 0))
    for kw in (dict(stream=None), dict(stream=HERE)):
        assert DecodeLayer.convolve(lay, conv, **t, **kw) == 0
        assert not marks                         # (torch's own rule for the current stream)
    assert DecodeLayer.convolve(lay, conv, **t, stream=handle) == 0
    assert on(marks, t.values(), name)
    marks.clear()
    parents = i(1, 0)
    lay._layer = lay._bufs = None
    assert DecodeLayer.reorder(lay, parents, 2, stream=HERE) == 0 and not marks
    assert DecodeLayer.reorder(lay, parents, 2, stream=handle) == 0
    assert on(marks, [parents], name)


@pytest.mark.parametrize("handle,name", [(9, ("external", 9)), (0, "default")])
def test_tensors_of_one_selection(marks, monkeypatch, handle, name):
    search = BeamSearch(2, 3, 7, device="cpu")
    dev = types.SimpleNamespace(type="cuda", index=None)
    search.scores = types.SimpleNamespace(device=dev, shape=search.scores.shape, dtype=torch.float32, data_ptr=search.scores.data_ptr)
    monkeypatch.setattr(serving, "_rows", lambda *a: 7)
    logits, scores, ended = torch.zeros(6, 7), torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int32)
    monkeypatch.setattr(serving, "_on_device", lambda index, call, stream: call(HERE if stream is None else stream))
    own = [types.SimpleNamespace(device=dev, **{n: getattr(t, n) for n in ("shape", "dtype", "is_contiguous", "data_ptr")},
                                 record_stream=lambda st, t=t: marks.append((t.data_ptr(), st))) for t in (scores, ended)]
    assert search.select(logits, *own, stream=HERE) == 0 and not marks
    assert search.select(logits, *own, stream=handle) == 0
    assert on(marks, [logits, scores, ended], name)
