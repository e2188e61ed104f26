"""The prompt, state-cache and output-norm calls reject invalid arguments on
the host, before any launch (runs without a GPU: every call here fails
validation or has nothing to do), and the Python layer refuses tensors that a
kernel must not read."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

from ssm_decode_amd import abi
from ssm_decode_amd.serving import OutputNorm, Prompts, StateCache, group_norm

from .test_abi import FAKE, OK_OFF, _bufs, _layer


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from ssm_decode_amd.build import build
        build()
    return abi.load()


def gdn(**kw):
    return _layer(OK_OFF, **{"family": abi.SKSSM_GDN, **kw})      # H 4, dk 16, dv 32, fp32, batch 2


def prompts(**over):
    f = dict(q=FAKE, k=FAKE, v=FAKE, gate=FAKE, beta=FAKE, o=FAKE, q_stride=64, k_stride=64, v_stride=128,
             gate_stride=4, beta_stride=4, o_stride=128, tokens=5, nseq=2, seq_start=FAKE, seqs=FAKE,
             has_state=FAKE, prime=1, work=FAKE, work_bytes=1 << 40)
    f.update(over)
    return abi.sketchssm_prompts(**f)


def cache(**over):
    f = dict(codes=FAKE, scale=FAKE, slots=3, bits=8)
    f.update(over)
    return abi.sketchssm_state_cache(**f)


def norm(**over):
    f = dict(x=FAKE, gate=FAKE, y=FAKE, weight=FAKE, bias=FAKE, x_stride=128, gate_stride=128, y_stride=128,
             rows=3, groups=2, width=64, dtype=abi.SKSSM_F32, group_weights=0, centred=0,
             activation=abi.SKSSM_ACT_SILU, gate_first=0, eps=1e-5)
    f.update(over)
    return abi.sketchssm_norm(**f)


def test_struct_sizes_match_the_header():
    """The binding's structs have the layout that a C compiler gives the header's."""
    import shutil
    import subprocess
    import tempfile
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    names = ("sketchssm_prompts", "sketchssm_state_cache", "sketchssm_norm")
    lines = []
    for n in names:
        lines.append(f'printf("%zu", sizeof({n}));')
        lines += [f'printf(" %zu", offsetof({n}, {f}));' for f, _ in getattr(abi, n)._fields_]
        lines.append('printf("\\n");')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "a.c"), os.path.join(d, "a")
        with open(src, "w") as f:
            f.write('#include <stdio.h>\n#include <stddef.h>\n#include "sketchssm.h"\nint main(void) {\n'
                    + "\n".join(lines) + "\nreturn 0; }\n")
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    for n, line in zip(names, out):
        ty = getattr(abi, n)
        assert [int(x) for x in line.split()] == [C.sizeof(ty)] + [getattr(ty, f).offset for f, _ in ty._fields_], n


# ------------------------------------------------------------------- prompts
def test_prefill_nothing_to_do():
    assert abi.sketchssm_prefill(gdn(), _bufs(), prompts(nseq=0, tokens=0, q=None, seq_start=None)) == 0


@pytest.mark.parametrize("field", ["q", "k", "v", "o", "gate", "beta", "seq_start"])
def test_prefill_null_and_misaligned(field):
    assert abi.sketchssm_prefill(gdn(), _bufs(), prompts(**{field: None})) == abi.SKSSM_EINVAL
    assert abi.sketchssm_prefill(gdn(), _bufs(), prompts(**{field: FAKE + 2})) == abi.SKSSM_EINVAL
    if field in "qkvo":
        assert abi.sketchssm_prefill(gdn(), _bufs(), prompts(**{field: FAKE + 8})) == abi.SKSSM_EINVAL


@pytest.mark.parametrize("field", ["seqs", "has_state"])
def test_prefill_misaligned_lists(field):
    assert abi.sketchssm_prefill(gdn(), _bufs(), prompts(**{field: FAKE + 1})) == abi.SKSSM_EINVAL


@pytest.mark.parametrize("field", ["S", "count", "err", "U", "Pt", "rank_offsets"])
def test_prefill_buffers(field):
    assert abi.sketchssm_prefill(gdn(), _bufs(**{field: None}), prompts()) == abi.SKSSM_EINVAL
    assert abi.sketchssm_prefill(gdn(), _bufs(**{field: FAKE + 4}), prompts()) == abi.SKSSM_EINVAL
    assert abi.sketchssm_prefill(gdn(), None, prompts()) == abi.SKSSM_EINVAL
    assert abi.sketchssm_prefill(gdn(), _bufs(), None) == abi.SKSSM_EINVAL
    assert abi.sketchssm_prefill(None, _bufs(), prompts()) == abi.SKSSM_EINVAL


def test_prefill_dense_heads_need_their_copies():
    L = _layer([0, 4, 4, 8, 12], family=abi.SKSSM_GDN)
    assert abi.sketchssm_prefill(L, _bufs(Scopy=None), prompts()) == abi.SKSSM_EINVAL


@pytest.mark.parametrize("over,code", [
    (dict(tokens=-1), abi.SKSSM_EDIM), (dict(nseq=-1), abi.SKSSM_EDIM), (dict(nseq=3), abi.SKSSM_EDIM),
    (dict(q_stride=60), abi.SKSSM_EDIM), (dict(q_stride=66), abi.SKSSM_EDIM), (dict(k_stride=0), abi.SKSSM_EDIM),
    (dict(v_stride=-128), abi.SKSSM_EDIM), (dict(o_stride=124), abi.SKSSM_EDIM), (dict(gate_stride=3), abi.SKSSM_EDIM),
    (dict(beta_stride=0), abi.SKSSM_EDIM), (dict(beta_stride=(1 << 25) + 4), abi.SKSSM_EDIM),
    (dict(q_stride=(1 << 25) + 64), abi.SKSSM_EDIM), (dict(prime=2), abi.SKSSM_EFLAG), (dict(prime=-1), abi.SKSSM_EFLAG),
])
def test_prefill_sizes_and_flags(over, code):
    assert abi.sketchssm_prefill(gdn(), _bufs(), prompts(**over)) == code


def test_prefill_families_and_maps():
    for fam in (abi.SKSSM_MAMBA2, abi.SKSSM_KDA):
        assert abi.sketchssm_prefill(_layer(OK_OFF, family=fam), _bufs(), prompts()) == abi.SKSSM_EDIM
    L = gdn(coef=abi.SKSSM_COEF_STATE, ridge=1e-4)
    assert abi.sketchssm_prefill(L, _bufs(), prompts()) == abi.SKSSM_EFLAG
    assert abi.sketchssm_prefill(L, _bufs(), prompts(prime=0, nseq=0)) == 0
    assert abi.sketchssm_prefill(gdn(W=0), _bufs(), prompts()) == abi.SKSSM_EDIM


def test_prefill_workspace():
    assert abi.sketchssm_prefill_workspace_bytes(gdn(), -1, 1) == abi.SKSSM_EDIM
    assert abi.sketchssm_prefill_workspace_bytes(gdn(), 1, 3) == abi.SKSSM_EDIM
    assert abi.sketchssm_prefill_workspace_bytes(None, 1, 1) == abi.SKSSM_EINVAL
    assert abi.sketchssm_prefill_workspace_bytes(_layer(OK_OFF), 1, 1) == abi.SKSSM_EDIM
    assert abi.sketchssm_prefill_workspace_bytes(gdn(), 0, 0) == 0
    # the chunked form (dk = 64: more than 48 tokens): a slot for every 64 tokens
    # and one for every prompt, 30.5 KiB for each of its heads, and 0.5 KiB
    L = gdn(dk=64, dv=64, act=abi.SKSSM_BF16, sk=abi.SKSSM_BF16)
    assert abi.sketchssm_prefill_workspace_bytes(L, 48, 2) == 0
    assert abi.sketchssm_prefill_workspace_bytes(L, 49, 2) == 0                        # 48 and 1
    assert abi.sketchssm_prefill_workspace_bytes(L, 50, 2) == 1 * 4 * 31232 + 512      # one prompt of 49 at most
    # fp32: 20.5 KiB; dk = 128: more than 24 tokens (fp32: 32)
    F = gdn(dk=64, dv=64)
    assert abi.sketchssm_prefill_workspace_bytes(F, 48, 2) == 0
    assert abi.sketchssm_prefill_workspace_bytes(F, 640, 2) == 12 * 4 * 20992 + 512
    assert abi.sketchssm_prefill_workspace_bytes(F, 1 << 17, 2) == (2048 + 2) * 4 * 20992 + 512
    for act, short in ((abi.SKSSM_BF16, 24), (abi.SKSSM_F32, 32)):
        G = gdn(dk=128, dv=64, act=act, sk=act)
        assert abi.sketchssm_prefill_workspace_bytes(G, short + 1, 2) == 0
        assert abi.sketchssm_prefill_workspace_bytes(G, short + 2, 2) > 0
    assert abi.sketchssm_prefill_workspace_bytes(L, 128, 2) == 4 * 4 * 31232 + 512
    assert abi.sketchssm_prefill_workspace_bytes(L, 640, 2) == 12 * 4 * 31232 + 512
    # few tiles with many tokens: also a state and a transition (fp32) for each
    # slot of 512 tokens or more and head, at most 48 to a prompt on average
    need = lambda t, n, shift: -(-((t // 64 + n) * 4 * 31232 + 512) // 256) * 256 + ((t >> shift) + n) * 4 * 64 * 128 * 4  # noqa: E731
    assert abi.sketchssm_prefill_workspace_bytes(L, 4095, 2) == (63 + 2) * 4 * 31232 + 512
    assert abi.sketchssm_prefill_workspace_bytes(L, 4096, 2) == need(4096, 2, 9)
    assert abi.sketchssm_prefill_workspace_bytes(L, 1 << 17, 2) == need(1 << 17, 2, 11)
    assert abi.sketchssm_prefill_workspace_bytes(L, 1 << 25, 2) == need(1 << 25, 2, 19)
    # at most 2^22 - 1 chunks of heads, prompts of heads, or entries of heads
    assert abi.sketchssm_prefill_workspace_bytes(L, 1 << 26, 2) == abi.SKSSM_EDIM
    assert abi.sketchssm_prefill_workspace_bytes(gdn(batch=1 << 20), 1 << 20, 1 << 20) == abi.SKSSM_EDIM
    assert abi.sketchssm_prefill_workspace_bytes(gdn(), 640, 2) == 0
    big = _layer(np.arange(129) * 4, family=abi.SKSSM_GDN, heads=128, groups=128, dk=64, dv=64, act=abi.SKSSM_BF16,
                 sk=abi.SKSSM_BF16)
    assert abi.sketchssm_prefill_workspace_bytes(big, (1 << 31) - 1, 2) == abi.SKSSM_EDIM
    strides = dict(q_stride=256, k_stride=256, v_stride=256, o_stride=256, tokens=640)
    for bad in (dict(work=None), dict(work=FAKE + 8), dict(work_bytes=12 * 4 * 31232 + 511)):
        assert abi.sketchssm_prefill(L, _bufs(), prompts(**strides, **bad)) == abi.SKSSM_EINVAL


# --------------------------------------------------------------- state cache
def both(L, B, Ca, seqs=FAKE, slots=FAKE, n=2, prime=1):
    return [abi.sketchssm_state_save(L, B, Ca, seqs, slots, n),
            abi.sketchssm_state_load(L, B, Ca, seqs, slots, n, prime)]


def test_cache_calls():
    L = _layer(OK_OFF)
    assert both(L, _bufs(), cache(), n=0) == [0, 0]
    assert both(L, _bufs(), cache(), seqs=None, slots=None, n=0) == [0, 0]
    E = abi.SKSSM_EINVAL
    assert both(None, _bufs(), cache()) == [E, E]
    assert both(L, None, cache()) == [E, E]
    assert both(L, _bufs(), None) == [E, E]
    for bad in (None, FAKE + 2):
        assert both(L, _bufs(), cache(), seqs=bad) == [E, E]
        assert both(L, _bufs(), cache(), slots=bad) == [E, E]
    for f in ("codes", "scale"):
        for bad in (None, FAKE + 8):
            assert both(L, _bufs(), cache(**{f: bad})) == [E, E]
    for f in ("S", "count", "err"):
        for bad in (None, FAKE + 4):
            assert both(L, _bufs(**{f: bad}), cache()) == [E, E]
    assert both(L, _bufs(), cache(bits=5)) == [abi.SKSSM_EDTYPE] * 2
    assert both(L, _bufs(), cache(slots=-1)) == [abi.SKSSM_EDIM] * 2
    assert both(L, _bufs(), cache(), n=-1) == [abi.SKSSM_EDIM] * 2
    assert both(L, _bufs(), cache(), n=1 << 30) == [abi.SKSSM_EDIM] * 2
    assert both(_layer(OK_OFF, W=0), _bufs(), cache()) == [abi.SKSSM_EDIM] * 2
    load = lambda L, B, prime: abi.sketchssm_state_load(L, B, cache(), FAKE, FAKE, 2, prime)  # noqa: E731
    assert load(L, _bufs(), 2) == abi.SKSSM_EFLAG
    assert load(L, _bufs(U=None), 1) == E and load(L, _bufs(Pt=FAKE + 4), 1) == E
    assert load(L, _bufs(rank_offsets=None), 1) == E
    assert load(_layer([0, 4, 4, 8, 12]), _bufs(Scopy=None), 1) == E
    assert load(_layer(OK_OFF, coef=abi.SKSSM_COEF_STATE, ridge=1e-4), _bufs(), 1) == abi.SKSSM_EFLAG


# ---------------------------------------------------------------------- norm
@pytest.mark.parametrize("over,code", [
    (dict(x=None), abi.SKSSM_EINVAL), (dict(x=FAKE + 8), abi.SKSSM_EINVAL), (dict(y=None), abi.SKSSM_EINVAL),
    (dict(y=FAKE + 4), abi.SKSSM_EINVAL), (dict(gate=FAKE + 8), abi.SKSSM_EINVAL),
    (dict(weight=FAKE + 4), abi.SKSSM_EINVAL), (dict(bias=FAKE + 4), abi.SKSSM_EINVAL),
    (dict(eps=-1.0), abi.SKSSM_EINVAL), (dict(eps=float("nan")), abi.SKSSM_EINVAL),
    (dict(eps=float("inf")), abi.SKSSM_EINVAL), (dict(rows=-1), abi.SKSSM_EDIM), (dict(groups=0), abi.SKSSM_EDIM),
    (dict(groups=65536, width=8), abi.SKSSM_EDIM), (dict(width=0), abi.SKSSM_EDIM), (dict(width=12), abi.SKSSM_EDIM),
    (dict(width=8200), abi.SKSSM_EDIM), (dict(x_stride=124), abi.SKSSM_EDIM), (dict(x_stride=130), abi.SKSSM_EDIM),
    (dict(y_stride=-128), abi.SKSSM_EDIM), (dict(gate_stride=0), abi.SKSSM_EDIM),
    (dict(y_stride=(1 << 25) + 64), abi.SKSSM_EDIM), (dict(dtype=2), abi.SKSSM_EDTYPE), (dict(dtype=-1), abi.SKSSM_EDTYPE),
    (dict(activation=3), abi.SKSSM_EFLAG), (dict(activation=-1), abi.SKSSM_EFLAG), (dict(centred=2), abi.SKSSM_EFLAG),
    (dict(gate_first=-1), abi.SKSSM_EFLAG), (dict(group_weights=2), abi.SKSSM_EFLAG),
])
def test_norm_refusals(over, code):
    assert abi.sketchssm_group_norm(norm(**over)) == code


def test_norm_nothing_to_do():
    assert abi.sketchssm_group_norm(norm(rows=0, x=None, y=None)) == 0
    assert abi.sketchssm_group_norm(None) == abi.SKSSM_EINVAL


# -------------------------------------------------------------- Python layer
class _Layer:
    """What Prompts and StateCache look at of a layer, on the CPU."""
    family, act, B, H, dk, dv = "gdn", "f32", 2, 4, 16, 32
    S = torch.zeros(2, 4, 16, 32)
    layer_struct = gdn()


def _tokens(N=5, **over):
    f = dict(q=torch.zeros(N, 4, 16), k=torch.zeros(N, 4, 16), v=torch.zeros(N, 4, 32), gate=torch.zeros(N, 4),
             beta=torch.zeros(N, 4), o=torch.zeros(N, 4, 32), seq_start=torch.tensor([0, 2, 5], dtype=torch.int32))
    f.update(over)
    return f


def test_prompts_take_strided_rows():
    rows = torch.zeros(5, 64 + 64 + 128 + 8)
    p = Prompts(_Layer(), **_tokens(q=rows[:, :64].unflatten(1, (4, 16)), k=rows[:, 64:128].unflatten(1, (4, 16)),
                                    v=rows[:, 128:256].unflatten(1, (4, 32))))
    assert (p.struct.q_stride, p.struct.v_stride, p.struct.o_stride, p.struct.gate_stride) == (264, 264, 128, 4)
    assert (p.struct.tokens, p.struct.nseq) == (5, 2)
    one = Prompts(_Layer(), **_tokens(1, seq_start=torch.tensor([0, 1], dtype=torch.int32)))
    assert one.struct.q_stride == 64


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(5, 4, 17)), dict(k=torch.zeros(4, 4, 16)), dict(v=torch.zeros(5, 4, 32, dtype=torch.bfloat16)),
    dict(q=torch.zeros(5, 16, 4).transpose(1, 2)), dict(gate=torch.zeros(4, 5).T), dict(beta=torch.zeros(5, 4, dtype=torch.float64)),
    dict(o=torch.zeros(5, 4, 64)[..., ::2]), dict(seq_start=torch.tensor([0, 2, 5])),
    dict(seq_start=torch.zeros(0, dtype=torch.int32)), dict(seq_start=torch.zeros(4, dtype=torch.int32)),
    dict(seqs=torch.zeros(3, dtype=torch.int32)), dict(seqs=torch.zeros(2)),
    dict(has_state=torch.zeros(4, dtype=torch.int32)[::2]), dict(q=torch.zeros(5, 4, 16, device="meta")),
])
def test_prompts_refuse_wrong_tensors(over):
    with pytest.raises(ValueError):
        Prompts(_Layer(), **_tokens(**over))


def test_prompts_belong_to_layers_of_their_shape():
    p = Prompts(_Layer(), **_tokens())
    p.check(_Layer())
    for name, value in (("H", 5), ("B", 3), ("dk", 64), ("dv", 64), ("act", "bf16"), ("family", "kda"),
                        ("S", torch.zeros(1, device="meta"))):
        other = type("Other", (_Layer,), {name: value})
        with pytest.raises(ValueError):
            p.check(other())


def test_prompts_refuse_norms_that_do_not_fit():
    z = torch.zeros(5, 4, 32)
    Prompts(_Layer(), **_tokens(), norm=OutputNorm(torch.ones(4, 32)), norm_gate=z)
    Prompts(_Layer(), **_tokens(), norm=OutputNorm(torch.ones(32)))
    for kw in (dict(norm=OutputNorm(torch.ones(4, 16))), dict(norm=OutputNorm(None, torch.ones(5, 32))),
               dict(norm=OutputNorm(torch.ones(32, device="meta"))), dict(norm_gate=z),
               dict(norm=OutputNorm(), norm_gate=z[:4])):
        with pytest.raises(ValueError):
            Prompts(_Layer(), **_tokens(), **kw)


def test_state_cache_refuses_wrong_entries():
    with pytest.raises(ValueError):
        StateCache(_Layer(), 2, 5)
    with pytest.raises(ValueError):
        StateCache(_Layer(), -1)
    c = StateCache(_Layer(), 2, 4)
    assert tuple(c.codes.shape) == (2, 4, 16, 16) and tuple(c.scale.shape) == (2, 4, 16, 1)
    i = torch.zeros(2, dtype=torch.int32)
    c.check(_Layer(), i, i)
    for a, b in ((i, i[:1]), (i.long(), i), (i, torch.zeros(4, dtype=torch.int32)[::2]), (i, i.to("meta"))):
        with pytest.raises(ValueError):
            c.check(_Layer(), a, b)

    class Other(_Layer):
        dv = 64
    with pytest.raises(ValueError):
        c.check(Other(), i, i)


def test_output_norm_refuses_wrong_tensors():
    for kw in (dict(weight=torch.zeros(4, dtype=torch.float64)), dict(weight=torch.zeros(4, 8).T), dict(act="relu"),
               dict(weight=torch.zeros(8), bias=torch.zeros(2, 8)), dict(bias=torch.zeros(1, 2, 3))):
        with pytest.raises(ValueError):
            OutputNorm(**kw)
    x = torch.zeros(3, 2, 8)
    with pytest.raises(ValueError):
        group_norm(x, OutputNorm(), x)                   # host memory


def test_prompts_refuse_norms_that_the_call_would_refuse():
    """What sketchssm_group_norm would refuse behind the prompts, whose states
    would then have moved on."""
    for eps in (float("nan"), float("inf"), -1e-5, 1e39):
        with pytest.raises(ValueError):
            OutputNorm(eps=eps)
    ok = torch.zeros(2000)
    at = next(i for i in range(4) if (ok.data_ptr() + 4 * i) % 16 == 0)
    w = ok[at + 1:at + 33]
    rows = ok[at:at + 5 * 132].view(5, 132)[:, :128].unflatten(1, (4, 32))
    Prompts(_Layer(), **_tokens(), norm=OutputNorm(ok[at:at + 32]), norm_gate=rows)
    odd = torch.zeros(5, 130)[:, :128].unflatten(1, (4, 32))
    for kw in (dict(norm=OutputNorm(w)), dict(norm=OutputNorm(None, w)), dict(norm=OutputNorm(), norm_gate=odd),
               dict(norm=OutputNorm(), norm_gate=ok[at + 1:at + 641].view(5, 4, 32)),
               dict(norm=OutputNorm(), norm_gate=torch.zeros(1, 4, 32).expand(5, 4, 32))):
        with pytest.raises(ValueError):
            Prompts(_Layer(), **_tokens(), **kw)
