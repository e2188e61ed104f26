"""A Mamba-2 layer's serving loop in small: a prompt through the convolution and the
scan, its state forked to the request's beams, then decode steps through the
convolution, the read and the flush, with the selection's parents reordering the
sequences behind each; against the recurrence in 64 bits, followed along the beams
that were selected."""
import numpy as np
import pytest
import torch

from tests import sequence_ref as ref

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.layer import DecodeLayer, TORCH_DTYPE
    from ssm_decode_amd.serving import BeamSearch, ScanPrompts, ShortConv


def f64(x):
    return x.double().cpu().numpy()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("act,tol", [("f32", 3e-5), ("bf16", 2.0 ** -6)])
def test_beam_search(act, tol):
    """tol, relative to each compared tensor's norm: fp32, the recurrence's roundings
    (below 1e-5) and the decode path's decays (2^-16); bf16, one rounding of the
    convolution's outputs (2^-8 each of q, k and v) and of o.  Head 1 reads a
    copy of its state; the others' outputs are compared where the flush gives
    them exactly."""
    n, k, H, G, dk, dv, W, V = 2, 3, 4, 2, 64, 64, 4, 50
    B, d = n * k, TORCH_DTYPE[act]
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    lay = DecodeLayer("mamba2", B, H, G, dk, dv, W, act, act, np.array([0, 8, 8, 16, 24]))
    lay.Pt.copy_(rand(24, dk) / 8)
    lay.Cmap.copy_(lay.Pt)
    lay.A.copy_(torch.log(1 + 7 * torch.rand(H, generator=g, device="cuda")))
    C = 2 * G * dk + H * dv
    conv = ShortConv(lay, rand(C, 4) / 2, 0.1 * rand(C))
    embed, steps_dt = rand(V, C).to(d), (0.01 + 0.09 * torch.rand((V, H), generator=g, device="cuda")).to(d)
    unembed = rand(H * dv, V) / 4
    search = BeamSearch(n, k, V, end=V - 1)
    w, b, A = f64(conv.weight), f64(conv.bias), f64(lay.A)

    def split(y):
        y = torch.from_numpy(y).to(d).double().numpy() if act == "bf16" else y
        return y[:, H * dv + G * dk:].reshape(-1, G, dk), y[:, H * dv:H * dv + G * dk].reshape(-1, G, dk), y[:, :H * dv].reshape(-1, H, dv)

    def run(tokens):
        """o of every token of a sequence, and its state, from its tokens alone."""
        y = ref.conv(f64(embed)[tokens], np.zeros((3, C)), w, b, "silu")[1]
        q, kk, v = split(y)
        o, S, _, _ = ref.scan(q, kk, v, f64(steps_dt)[tokens], A, np.zeros((H, dk, dv)))
        return o, S

    # a request's prompt goes to its first beam, which the others are copies of
    prompts = [torch.randint(0, V - 1, (t,), generator=g, device="cuda") for t in (41, 150)]
    tok = torch.cat(prompts)
    start, seqs = ints(0, 41, 191), ints(0, k)
    y = torch.empty(191, C, device="cuda", dtype=d)
    q, kk, v = (y[:, H * dv + G * dk:].unflatten(1, (G, dk)), y[:, H * dv:H * dv + G * dk].unflatten(1, (G, dk)),
                y[:, :H * dv].unflatten(1, (H, dv)))
    fresh = ints(0, 0)
    assert lay.convolve(conv, embed[tok], q, kk, v, seq_start=start, seqs=seqs, has_state=fresh) == 0
    o = torch.empty(191, H, dv, device="cuda", dtype=d)
    assert lay.scan(ScanPrompts(lay, q, kk, v, steps_dt[tok], o, start, seqs, fresh)) == 0
    assert lay.reorder(ints(0, 0, 0, 3, 3, 3), k, convs=(conv,)) == 0
    paths = [prompts[i // k].tolist() for i in range(B)]
    outs = torch.stack([o[40], o[190]]).repeat_interleave(k, 0)
    for i, p in enumerate(paths):
        want, S = run(p)
        assert np.linalg.norm(f64(lay.S[i]) - S) <= tol * np.linalg.norm(S)
        assert np.linalg.norm(f64(outs[i]) - want[-1]) <= tol * np.linalg.norm(want[-1])

    for t in range(2 * W):
        logits = outs.flatten(1).float() @ unembed
        before, s, e = paths, search.scores.clone(), search.ended.clone()
        assert search.select(logits) == 0
        parents, tokens, scores, _ = ref.beams(f64(logits).reshape(n, k, V), f64(s), e.cpu().numpy(), V - 1)
        assert (search.parents.cpu().numpy() == parents).all() and (search.tokens.cpu().numpy() == tokens).all()
        assert lay.reorder(search.parents, k, convs=(conv,)) == 0
        x = search.tokens.flatten().long()
        step = lay.new_step()
        assert lay.convolve(conv, embed[x], step.q, step.k, step.v) == 0
        step.gate.copy_(steps_dt[x])
        assert lay.read(step) == 0 and lay.flush(step) == 0
        paths = [before[p] + [int(c)] for p, c in zip(parents.flatten(), tokens.flatten())]
        outs = step.o
        if t % W == W - 1:
            for i, p in enumerate(paths):
                want, S = run(p)
                assert np.linalg.norm(f64(lay.S[i]) - S) <= tol * np.linalg.norm(S)
                assert np.linalg.norm(f64(outs[i]) - want[-1]) <= tol * np.linalg.norm(want[-1])
    assert lay.error_word() == 0 and conv.error_word() == 0 and search.error_word() == 0
