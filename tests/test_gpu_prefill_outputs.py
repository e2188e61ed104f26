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


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 32), (64, 64), (128, 64), (128, 128)])
def test_single_tokens_agree_with_the_decode_step(act, dk, dv):
    """A token through sketchssm_prefill and through sketchssm_full_step: each
    is off by at most (dk + 8) roundings of 2^-24 of the column's norm (the sum
    over a column, the update, the output), the outputs by half a step more."""
    B, H = 5, 3
    lay, other = (make_layer(B, H, dk, dv, act, seed=360) for _ in range(2))
    tok = make_tokens(B, H, dk, dv, act, seed=361)
    S0 = lay.S.clone()
    run(lay, tok, [1] * B)
    st = other.new_step()
    for dst, src in zip((st.q, st.k, st.v, st.gate, st.beta), tok):
        dst.copy_(src)
    assert other.full_step(st) == 0
    torch.cuda.synchronize()
    assert lay.error_word() == other.error_word() == 0
    for b in range(B):
        o, S, scale = rule(*(x[b:b + 1] for x in tok[:5]), S0[b])
        column = torch.maximum(S.norm(dim=1, keepdim=True), S0[b].double().norm(dim=1, keepdim=True))
        noise = (dk + 8) * 2.0 ** -24
        assert ((lay.S[b].double() - other.S[b].double()).abs() <= 2 * noise * column).all()
        lim = 2 * noise * column[:, 0] * tok[0][b].double().norm(dim=-1, keepdim=True)
        lim = lim + torch.finfo(tok[5].dtype).eps * (o[0].abs() + lim)
        assert ((tok[5][b].double() - st.o[b].double()).abs() <= lim).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[2300], [300, 90], [9, 3]], ids=lambda x: "-".join(map(str, x)))
def test_two_calls_at_once_on_one_layer(act, lens):
    """Disjoint sequences of one layer, a stream and a ``Prompts`` each, again and
    again."""
    n, N = len(lens), sum(lens)
    lay = make_layer(2 * n + 1, 3, 128, 128, act, seed=370)
    toks = [make_tokens(N, 3, 128, 128, act, seed=371 + i) for i in range(2)]
    starts = [sum(lens[:i]) for i in range(n + 1)]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    from ssm_decode_amd.serving import Prompts
    seqs = [list(range(0, 2 * n, 2)), list(range(1, 2 * n, 2))]
    prs = [Prompts(lay, *t, dev(starts), dev(s)) for t, s in zip(toks, seqs)]
    S0 = lay.S.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        lay.S.copy_(S0)
        for t in toks:
            t[5].fill_(SENTINEL)
        torch.cuda.synchronize()
        for st, p in zip(streams, prs):
            assert lay.prefill(p, stream=st.cuda_stream) == 0
        torch.cuda.synchronize()
        assert lay.error_word() == 0
        for t, s in zip(toks, seqs):
            for i in range(n):
                part = slice(starts[i], starts[i + 1])
                o, S, scale = rule(*(x[part] for x in t[:5]), S0[s[i]])
                assert wrong_outputs(t[5][part], o, scale, 128) == (0, 0)
                assert state_off(lay.S[s[i]], S, 128) == 0
        assert torch.equal(lay.S[2 * n], S0[2 * n])
