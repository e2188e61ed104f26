"""The scan, convolution, beam and reordering calls reject invalid arguments on the
host, before any launch (no GPU: every call here fails validation or has nothing to
do), and the Python layer refuses tensors that a kernel must not read."""
import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

from ssm_decode_amd import abi
from ssm_decode_amd.layer import DecodeLayer
from ssm_decode_amd.serving import BeamSearch, ScanPrompts, ShortConv

from .test_abi import FAKE, OK_OFF, _bufs, _layer

E, D, T, F = abi.SKSSM_EINVAL, abi.SKSSM_EDIM, abi.SKSSM_EDTYPE, abi.SKSSM_EFLAG


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from ssm_decode_amd.build import build
        build()
    return abi.load()


def m2(**kw):
    return _layer(OK_OFF, **kw)                       # H 4, dk 16, dv 32, fp32, batch 2


def test_struct_sizes_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    names = ("sketchssm_scan_prompts", "sketchssm_conv_piece", "sketchssm_convolution", "sketchssm_beams", "sketchssm_rows")
    lines = []
    for n in names:
        lines.append(f'printf("%zu", sizeof({n}));')
        lines += [f'printf(" %zu", offsetof({n}, {f}));' for f, _ in getattr(abi, n)._fields_]
        lines.append('printf("\\n");')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "a.c", tmp_path / "a"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "sketchssm.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    for n, line in zip(names, out):
        ty = getattr(abi, n)
        assert [int(x) for x in line.split()] == [C.sizeof(ty)] + [getattr(ty, f).offset for f, _ in ty._fields_], n


# ---------------------------------------------------------------------- scan
def scan(**over):
    f = dict(q=FAKE, k=FAKE, v=FAKE, dt=FAKE, o=FAKE, q_stride=64, k_stride=64, v_stride=128, dt_stride=4, o_stride=128,
             tokens=5, nseq=2, seq_start=FAKE, seqs=FAKE, has_state=FAKE, prime=1, work=FAKE, work_bytes=1 << 40)
    f.update(over)
    return abi.sketchssm_scan_prompts(**f)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), E), (dict(k=FAKE + 8), E), (dict(v=None), E), (dict(o=FAKE + 4), E), (dict(dt=None), E), (dict(dt=FAKE + 2), E),
    (dict(seq_start=None), E), (dict(seqs=FAKE + 2), E), (dict(has_state=FAKE + 1), E), (dict(tokens=-1), D), (dict(nseq=-1), D),
    (dict(nseq=3), D), (dict(q_stride=60), D), (dict(k_stride=66), D), (dict(v_stride=124), D), (dict(o_stride=-128), D),
    (dict(dt_stride=3), D), (dict(dt_stride=(1 << 25) + 1), D), (dict(q_stride=(1 << 25) + 64), D), (dict(prime=2), F), (dict(prime=-1), F),
])
def test_scan_refusals(over, code):
    assert abi.sketchssm_scan(m2(), _bufs(), scan(**over)) == code


@pytest.mark.parametrize("field", ["S", "count", "err", "A", "U", "Pt", "rank_offsets"])
def test_scan_buffers(field):
    assert abi.sketchssm_scan(m2(), _bufs(**{field: None}), scan()) == E
    assert abi.sketchssm_scan(m2(), _bufs(**{field: FAKE + 4}), scan()) == E


def test_scan_layers():
    for fam in (abi.SKSSM_GDN, abi.SKSSM_KDA):
        assert abi.sketchssm_scan(m2(family=fam), _bufs(), scan()) == D
        assert abi.sketchssm_scan_workspace_bytes(m2(family=fam), 1, 1) == D
    assert abi.sketchssm_scan(None, _bufs(), scan()) == E and abi.sketchssm_scan(m2(), None, scan()) == E
    assert abi.sketchssm_scan(m2(), _bufs(), None) == E
    assert abi.sketchssm_scan(_layer([0, 4, 4, 8, 12]), _bufs(Scopy=None), scan()) == E
    L = m2(coef=abi.SKSSM_COEF_STATE, ridge=1e-4)
    assert abi.sketchssm_scan(L, _bufs(), scan()) == F and abi.sketchssm_scan(L, _bufs(), scan(prime=0, nseq=0)) == 0
    assert abi.sketchssm_scan(m2(), _bufs(), scan(nseq=0, tokens=0, q=None, seq_start=None)) == 0
    assert abi.sketchssm_scan_workspace_bytes(m2(), -1, 1) == D and abi.sketchssm_scan_workspace_bytes(m2(), 1, 3) == D
    assert abi.sketchssm_scan_workspace_bytes(None, 1, 1) == E and abi.sketchssm_scan_workspace_bytes(m2(), 0, 0) == 0
    assert abi.sketchssm_scan_workspace_bytes(m2(batch=1 << 21), 1 << 21, 1 << 21) == D


# --------------------------------------------------------------- convolution
def conv(pieces=((64, 0), (64, 64), (128, 16)), **over):
    f = dict(x=FAKE, x_stride=256, weight=FAKE, bias=FAKE, state=FAKE, taps=4, dtype=abi.SKSSM_F32,
             activation=abi.SKSSM_ACT_SILU, eps=1e-6, batch=3, tokens=5, nseq=2, seq_start=FAKE, seqs=FAKE, has_state=FAKE, err=FAKE)
    f.update(over)
    p = [abi.sketchssm_conv_piece(x[2] if len(x) > 2 else FAKE, x[3] if len(x) > 3 else max(x[0], 1), x[0], x[1]) for x in pieces]
    return abi.sketchssm_conv(abi.sketchssm_convolution(piece=(abi.sketchssm_conv_piece * 3)(*p), **f))


@pytest.mark.parametrize("over,code", [
    (dict(x=None), E), (dict(x=FAKE + 8), E), (dict(weight=None), E), (dict(weight=FAKE + 4), E), (dict(bias=FAKE + 4), E),
    (dict(state=None), E), (dict(state=FAKE + 8), E), (dict(err=None), E), (dict(seq_start=FAKE + 2), E), (dict(seqs=FAKE + 2), E),
    (dict(has_state=FAKE + 2), E), (dict(taps=1), D), (dict(taps=9), D), (dict(dtype=2), T), (dict(dtype=-1), T),
    (dict(activation=3), F), (dict(activation=-1), F), (dict(eps=-1.0), E), (dict(eps=float("nan")), E), (dict(eps=float("inf")), E),
    (dict(batch=1), D), (dict(batch=-1, nseq=-2), D), (dict(tokens=-1), D), (dict(nseq=-1), D), (dict(seq_start=None), D),
    (dict(x_stride=252), D), (dict(x_stride=258), D), (dict(x_stride=(1 << 25) + 256), D),
    (dict(pieces=((-8, 0), (64, 0), (64, 0))), D), (dict(pieces=((60, 0), (64, 0), (64, 0))), D), (dict(pieces=((64, 32), (64, 0), (64, 0))), D),
    (dict(pieces=((64, 128), (64, 0), (64, 0))), D), (dict(pieces=((64, 0, None), (64, 0), (64, 0))), E),
    (dict(pieces=((64, 0, FAKE + 8), (64, 0), (64, 0))), E), (dict(pieces=((64, 0, FAKE, 60), (64, 0), (64, 0))), D),
    (dict(pieces=((1 << 25, 0), (64, 0), (64, 0))), D),
])
def test_conv_refusals(over, code):
    assert conv(**over) == code


def test_conv_nothing_to_do():
    assert conv(nseq=0, tokens=0, x=None, state=None, seq_start=None) == 0
    assert conv(pieces=((0, 0), (0, 0), (0, 0))) == 0
    assert abi.sketchssm_conv(None) == E


# --------------------------------------------------------------------- beams
def beams(**over):
    f = dict(logits=FAKE, stride=100, scores=FAKE, ended=FAKE, new_scores=FAKE, new_ended=FAKE, parents=FAKE, tokens=FAKE, err=FAKE,
             groups=2, beams=4, vocab=100, dtype=abi.SKSSM_BF16, end_token=3, work=FAKE, work_bytes=1 << 40)
    f.update(over)
    return abi.sketchssm_beam_select(abi.sketchssm_beams(**f))


@pytest.mark.parametrize("over,code", [
    (dict(logits=None), E), (dict(logits=FAKE + 1), E), (dict(scores=None), E), (dict(scores=FAKE + 2), E), (dict(ended=FAKE + 2), E),
    (dict(new_scores=None), E), (dict(new_ended=None), E), (dict(parents=FAKE + 2), E), (dict(tokens=None), E), (dict(err=None), E),
    (dict(work=None), E), (dict(work=FAKE + 8), E), (dict(work_bytes=10), E), (dict(stride=99), D), (dict(stride=1 << 31), D),
    (dict(groups=-1), D), (dict(beams=0), D), (dict(beams=17), D), (dict(vocab=0), D), (dict(vocab=(1 << 24) + 1, stride=1 << 25), D),
    (dict(end_token=-2), D), (dict(end_token=100), D), (dict(dtype=2), T), (dict(dtype=-1), T), (dict(groups=1 << 30), D),
])
def test_beam_refusals(over, code):
    assert beams(**over) == code


def test_beam_nothing_to_do():
    assert beams(groups=0, logits=None, work=None) == 0
    assert abi.sketchssm_beam_select(None) == E
    assert abi.sketchssm_beam_workspace_bytes(1, 1, 1, 5) == T and abi.sketchssm_beam_workspace_bytes(-1, 1, 1, 0) == D
    assert abi.sketchssm_beam_workspace_bytes(0, 4, 100, 0) == 0


# ---------------------------------------------------------------- reordering
def rows(*x):
    return (abi.sketchssm_rows * max(1, len(x)))(*(abi.sketchssm_rows(*y) for y in x))


def test_reorder_refusals():
    call = lambda L=None, B=None, x=(), n=None, parents=FAKE, k=2: abi.sketchssm_reorder(  # noqa: E731
        L or m2(), _bufs() if B is None else B, rows(*x), len(x) if n is None else n, parents, k)
    for k in (0, -1, 17, 3):
        assert call(k=k) == D
    assert call(parents=None) == E and call(parents=FAKE + 2) == E and call(n=-1) == D and call(n=5) == D
    assert abi.sketchssm_reorder(m2(), _bufs(), None, 1, FAKE, 2) == E
    assert abi.sketchssm_reorder(None, _bufs(), None, 0, FAKE, 2) == E and abi.sketchssm_reorder(m2(), None, None, 0, FAKE, 2) == E
    for name in ("S", "U", "ring_k", "ring_v", "ring_gate", "count", "err"):
        assert call(B=_bufs(**{name: None})) == E and call(B=_bufs(**{name: FAKE + 4})) == E, name
    assert call(x=((FAKE, 8),)) == D and call(x=((FAKE, -16),)) == D and call(x=((FAKE + 8, 16),)) == E and call(x=((None, 16),)) == E
    far = FAKE << 20                             # (rows listed twice, one behind the other's start, the layer's own)
    assert call(x=((far, 16), (far, 16))) == E and call(x=((far, 32), (far + 48, 16))) == E and call(x=((FAKE, 16),)) == E
    gdn = m2(family=abi.SKSSM_GDN)
    assert call(gdn, _bufs(ring_beta=None)) == E
    assert call(_layer([0, 4, 4, 8, 12]), _bufs(Scopy=None)) == E
    assert call(m2(coef=abi.SKSSM_COEF_STATE, ridge=1e-4), _bufs(Cstate=None)) == E
    assert call(m2(batch=0)) in (0, D)


# -------------------------------------------------------------- Python layer
class _Layer:
    """What the objects look at of a layer, on the CPU."""
    family, act, B, H, G, dk, dv = "mamba2", "f32", 2, 4, 4, 16, 32
    S = torch.zeros(2, 4, 16, 32)
    layer_struct = m2()


def _tokens(N=5, **over):
    f = dict(q=torch.zeros(N, 4, 16), k=torch.zeros(N, 4, 16), v=torch.zeros(N, 4, 32), dt=torch.zeros(N, 4),
             o=torch.zeros(N, 4, 32), seq_start=torch.tensor([0, 2, 5], dtype=torch.int32))
    f.update(over)
    return f


def test_scan_prompts_take_strided_rows():
    r = torch.zeros(5, 264)
    p = ScanPrompts(_Layer(), **_tokens(q=r[:, :64].unflatten(1, (4, 16)), v=r[:, 128:256].unflatten(1, (4, 32)), dt=r[:, 256:260]))
    assert (p.struct.q_stride, p.struct.k_stride, p.struct.v_stride, p.struct.dt_stride, p.struct.tokens, p.struct.nseq) == (264, 64, 264, 264, 5, 2)


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(5, 2, 16)), dict(k=torch.zeros(4, 4, 16)), dict(v=torch.zeros(5, 4, 32, dtype=torch.bfloat16)), dict(dt=torch.zeros(4, 5).T),
    dict(o=torch.zeros(5, 4, 64)[..., ::2]), dict(seq_start=torch.tensor([0, 2, 5])), dict(seq_start=torch.zeros(0, dtype=torch.int32)),
    dict(seq_start=torch.zeros(4, dtype=torch.int32)), dict(seqs=torch.zeros(3, dtype=torch.int32)), dict(has_state=torch.zeros(2)),
    dict(q=torch.zeros(5, 4, 16, device="meta")),
])
def test_scan_prompts_refuse_wrong_tensors(over):
    with pytest.raises(ValueError):
        ScanPrompts(_Layer(), **_tokens(**over))


def test_objects_belong_to_layers_of_their_shape():
    p, c = ScanPrompts(_Layer(), **_tokens()), ShortConv(_Layer(), torch.zeros(256, 4))
    p.check(_Layer())
    c.check(_Layer())
    for name, value in (("H", 5), ("B", 3), ("G", 2), ("dk", 64), ("dv", 64), ("act", "bf16"), ("family", "gdn"), ("S", torch.zeros(1, device="meta"))):
        other = type("Other", (_Layer,), {name: value})
        for x in (p, c):
            with pytest.raises(ValueError):
                x.check(other())


@pytest.mark.parametrize("kw", [
    dict(weight=torch.zeros(255, 4)), dict(weight=torch.zeros(256, 1)), dict(weight=torch.zeros(256, 9)), dict(weight=torch.zeros(4, 256).T),
    dict(weight=torch.zeros(256, 4, dtype=torch.bfloat16)), dict(bias=torch.zeros(255)), dict(bias=torch.zeros(512)[::2]), dict(act="relu"),
    dict(order="qk"), dict(order="qqv"), dict(eps=-1.0), dict(eps=float("nan")), dict(weight=torch.zeros(1025)[1:].view(256, 4)),
])
def test_short_conv_refuses_wrong_tensors(kw):
    with pytest.raises(ValueError):
        ShortConv(_Layer(), **dict(dict(weight=torch.zeros(256, 4)), **kw))


def test_convolve_refuses_wrong_tensors():
    c = ShortConv(_Layer(), torch.zeros(256, 4))
    ok = dict(x=torch.zeros(2, 256), q=torch.zeros(2, 4, 16), k=torch.zeros(2, 4, 16), v=torch.zeros(2, 4, 32))
    i = torch.zeros(2, dtype=torch.int32)
    for over in (dict(x=torch.zeros(2, 255)), dict(x=torch.zeros(256, 2).T), dict(q=torch.zeros(3, 4, 16)), dict(k=torch.zeros(2, 4, 17)),
                 dict(v=torch.zeros(2, 4, 32, dtype=torch.bfloat16)), dict(seqs=i[:1]), dict(has_state=i.long()), dict(seq_start=i.long()),
                 dict(seq_start=torch.zeros(4, dtype=torch.int32), seqs=i)):
        with pytest.raises(ValueError):
            DecodeLayer.convolve(_Layer(), c, **dict(ok, **over))
    lay = _Layer()
    for bad in (torch.zeros(3, dtype=torch.int32), torch.zeros(2), torch.zeros(4, dtype=torch.int32)[::2], i.to("meta")):
        with pytest.raises(ValueError):
            DecodeLayer.reorder(lay, bad, 2)
    with pytest.raises(ValueError):
        DecodeLayer.reorder(type("Other", (_Layer,), {"G": 2})(), i, 2, convs=(c,))


def test_beam_search_refuses_wrong_tensors():
    for a in ((-1, 2, 5), (1, 0, 5), (1, 17, 5), (1, 2, 0), (1, 2, (1 << 24) + 1), (1, 2, 5, 5), (1, 2, 5, -2), (1 << 26, 16, 5)):
        with pytest.raises(ValueError):
            BeamSearch(*a, device="cpu")
    s = BeamSearch(2, 3, 7, device="cpu")
    assert s.scores.tolist() == [[0.0, -float("inf"), -float("inf")]] * 2
    with pytest.raises(ValueError):
        s.select(torch.zeros(6, 7))                      # host memory
