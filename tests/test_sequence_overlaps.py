"""Outputs that share memory with what a call reads, or with each other, are refused:
one workgroup would read what another has written (no GPU)."""
import random

import pytest
import torch

from ssm_decode_amd import serving
from ssm_decode_amd.layer import DecodeLayer
from ssm_decode_amd.serving import ScanPrompts, ShortConv

from .test_sequence_abi import _Layer, _tokens, lib  # noqa: F401  (lib: the library is built)

H, G, DK, DV, N = 4, 4, 16, 32, 5


def cut(rows, first, heads, width):
    return rows[:, first:first + heads * width].unflatten(1, (heads, width))


def test_what_shares_memory():
    rng = random.Random(5)
    for _ in range(20000):
        spans, taken, n = [], [], rng.randint(0, 5)
        for _ in range(2):
            size = rng.randint(1, 12)
            stride = max(size, rng.choice((size, size + rng.randint(0, 20), 24, 25)))
            first = rng.randint(0, 60)
            spans.append((first, stride, size))
            taken.append({first + i * stride + e for i in range(n) for e in range(size)})
        assert serving._shared(spans, n) == ((0, 1) if taken[0] & taken[1] else None), (spans, n)


@pytest.mark.parametrize("name", ["v", "q", "k"])
def test_scan_outputs_over_inputs(name):
    t = _tokens()
    rows = torch.zeros(N, 4 * 32)
    t["o"] = rows.unflatten(1, (H, DV))
    t[name] = cut(rows, 0, H, DV) if name == "v" else cut(rows, 64, G, DK)
    with pytest.raises(ValueError, match="o shares"):
        ScanPrompts(_Layer(), **t)


def test_scan_outputs_partly_over_an_input():
    rows = torch.zeros(N + 2, 128)               # two rows on
    with pytest.raises(ValueError, match="o shares"):
        ScanPrompts(_Layer(), **_tokens(v=rows[:N].unflatten(1, (H, DV)), o=rows[2:].unflatten(1, (H, DV))))
    rows = torch.zeros(N, 264)                   # a column of dt in o's row
    with pytest.raises(ValueError, match="o shares"):
        ScanPrompts(_Layer(), **_tokens(o=cut(rows, 0, H, DV), dt=rows[:, 126:130]))


def test_scan_outputs_between_the_inputs():
    rows = torch.zeros(N, 400)
    p = ScanPrompts(_Layer(), **_tokens(q=cut(rows, 0, G, DK), k=cut(rows, 64, G, DK), o=cut(rows, 128, H, DV), v=cut(rows, 256, H, DV),
                                        dt=rows[:, 384:388]))
    assert p.struct.o_stride == 400
    # (the inputs may be one)
    t = _tokens()
    ScanPrompts(_Layer(), **dict(t, q=t["k"]))


@pytest.fixture
def convolve(monkeypatch):
    """The call up to the library's."""
    monkeypatch.setattr(serving, "_on_device", lambda index, call, stream: 0)
    conv = ShortConv(_Layer(), torch.zeros(256, 4))
    return lambda **kw: DecodeLayer.convolve(_Layer(), conv, **kw)


@pytest.mark.parametrize("prompts", [True, False])
def test_convolution_outputs(convolve, prompts):
    kw = dict(seq_start=torch.tensor([0, 2, 5], dtype=torch.int32)) if prompts else {}
    new = lambda c: torch.zeros(N, c)  # noqa: E731
    x = new(256)
    ok = dict(x=x, q=new(64).view(N, G, DK), k=new(64).view(N, G, DK), v=new(128).view(N, H, DV))
    assert convolve(**ok, **kw) == 0
    y, wide = new(256), new(600)
    out = lambda r, f: dict(v=cut(r, f, H, DV), k=cut(r, f + 128, G, DK), q=cut(r, f + 192, G, DK))  # noqa: E731
    assert convolve(x=x, **out(y, 0), **kw) == 0
    assert convolve(x=wide[:, :256], **out(wide, 256), **kw) == 0
    assert convolve(x=wide[:, 344:], **out(wide, 0), **kw) == 0
    for bad in (dict(x=x, **out(x, 0)),                                # in place
                dict(ok, q=cut(x, 0, G, DK)), dict(ok, k=cut(x, 192, G, DK)), dict(ok, v=cut(x, 100, H, DV)),
                dict(x=wide[:, 200:456], **out(wide, 0)),
                dict(ok, q=ok["k"]), dict(ok, v=cut(y, 0, H, DV), k=cut(y, 64, G, DK)), dict(ok, q=cut(y, 0, G, DK), v=cut(y, 48, H, DV))):
        with pytest.raises(ValueError, match="shares? memory"):
            convolve(**bad, **kw)
