"""Outputs of long prompts by bounds that do not grow with the prompt, and
prompts in segments with several heads."""
import numpy as np
import pytest
import torch

from tests.prompt_bounds import rule, state_off, wrong_outputs
from tests.test_gpu_prefill import SENTINEL, make_layer, make_tokens, run

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd import abi
    from ssm_decode_amd.layer import DecodeLayer


def segment_bytes(lay, tokens, n):
    """The workspace's part for segments' states (0: the prompts go whole)."""
    slots = tokens // 64 + n
    return max(0, abi.sketchssm_prefill_workspace_bytes(lay.layer_struct, tokens, n) - slots * lay.H * 31232 - 1024)


def verify(lay, S0, tok, lens, starts, seqs, has):
    for i, n in enumerate(lens):
        part = slice(starts[i], starts[i] + n)
        s0 = S0[seqs[i]] if has[i] else torch.zeros_like(S0[seqs[i]])
        o, S, scale = rule(*(x[part] for x in tok[:5]), s0)
        assert wrong_outputs(tok[5][part], o, scale, lay.dk) == (0, 0), i
        assert state_off(lay.S[seqs[i]], S, lay.dk) == 0, i
        if n == 0:
            assert torch.equal(lay.S[seqs[i]], s0)
    assert (tok[5][starts[-1]:].float() == torch.tensor(SENTINEL).to(tok[5].dtype).float()).all()
    others = [b for b in range(lay.B) if b not in seqs]
    assert torch.equal(lay.S[others], S0[others])


def long_prompts(H, dk, dv, act, lens, seed, decay):
    n = len(lens)
    lay = make_layer(n + 1, H, dk, dv, act, seed=seed, ranks=[(5 * h) % 8 for h in range(H)])
    tok = make_tokens(sum(lens), H, dk, dv, act, seed=seed + 1, packed=True, pad=2)
    tok[3][:] = 1 - (1 - tok[3]) * decay
    S0 = lay.S.clone()
    seqs, has = [n - i for i in range(n)], [(i + 1) % 2 for i in range(n)]
    _, starts = run(lay, tok, lens, seqs=seqs, has=has)
    assert lay.error_word() == 0
    return lay, S0, tok, starts, seqs, has


SEGMENTED = [(1, [12300, 5, 1]), (1, [511, 512, 513, 6700]), (2, [4096, 0, 5000]), (3, [1, 8200]), (4, [4097]),
             (5, [5300, 4400]), (8, [3000, 1100, 4300]), (16, [2048, 2049]), (32, [2500])]


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,lens", SEGMENTED, ids=lambda x: str(x) if isinstance(x, int) else "-".join(map(str, x)))
def test_segments_of_several_heads(dk, dv, H, lens):
    lay, *rest = long_prompts(H, dk, dv, "bf16", lens, 300 + H, 0.01)
    assert segment_bytes(lay, sum(lens), len(lens)) > 0
    S0, tok, starts, seqs, has = rest
    verify(lay, S0, tok, lens, starts, seqs, has)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 32), (64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[2500], [700, 1, 0, 40, 1300, 64, 65]], ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("decay", [0.01, 1.0])
def test_whole_prompts(act, dk, dv, lens, decay):
    H = 33 if act == "bf16" and len(lens) == 1 else 5
    lay, S0, tok, starts, seqs, has = long_prompts(H, dk, dv, act, lens, 340 + len(lens), decay)
    if act == "f32" or H * len(lens) > 32:
        assert segment_bytes(lay, sum(lens), len(lens)) == 0
    verify(lay, S0, tok, lens, starts, seqs, has)


@pytest.mark.parametrize("act,n", [("bf16", 3), ("bf16", 100), ("f32", 100), ("bf16", 9000)])
def test_outputs_of_the_last_of_very_many_states(act, n):
    """The first and the last of 2^17 + 8 sequences, whose states' offsets pass
    32 bits: their outputs."""
    B, dk, dv = (1 << 17) + 8, 128, 128
    lay = DecodeLayer("gdn", B, 1, 1, dk, dv, 1, act, act, np.array([0, 3], dtype=np.int32))
    g = torch.Generator(device="cuda").manual_seed(395)
    ends = [0, B - 1]
    for b in ends:
        lay.S[b] = 0.1 * torch.randn(lay.S[b].shape, generator=g, device="cuda")
    first = [lay.S[b].clone() for b in ends]
    tok = make_tokens(2 * n, 1, dk, dv, act, seed=396)
    tok[3][:] = 1 - (1 - tok[3]) * 0.01
    run(lay, tok, [n, n], seqs=ends)
    assert lay.error_word() == 0
    for i, b in enumerate(ends):
        o, S, scale = rule(*(x[i * n:(i + 1) * n] for x in tok[:5]), first[i])
        assert wrong_outputs(tok[5][i * n:(i + 1) * n], o, scale, dk) == (0, 0)
        assert state_off(lay.S[b], S, dk) == 0
