"""A serving loop in small: prompts with their normalised outputs, a sequence's
state parked and read back into another, decode steps with the norm behind
them, and further prompts that go on from decoded states; against the token
recurrence in 64 bits."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.layer import DecodeLayer, TORCH_DTYPE
    from ssm_decode_amd.serving import OutputNorm, Prompts, StateCache


def f64(x):
    return x.double().cpu().numpy()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("act,tol", [("f32", 2e-5), ("bf16", 2.0 ** -7)])
def test_serving_loop(act, tol):
    """tol, relative to each compared tensor's norm: fp32, the recurrence's
    roundings over the tokens (as in the prompts' own test, below 1e-5) and the
    norm's; bf16, one rounding of o (2^-8), one of y (2^-8)."""
    B, H, dk, dv, W = 4, 3, 64, 64, 4
    dt = TORCH_DTYPE[act]
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    lay = DecodeLayer("gdn", B, H, H, dk, dv, W, act, act, np.array([0, 8, 8, 16]))   # head 1: a state copy
    lay.Pt.copy_(rand(16, dk) / 8)
    lay.Cmap.copy_(lay.Pt)
    norm = OutputNorm(1 + 0.1 * rand(dv), eps=1e-5, act="silu")
    S = np.zeros((B, H, dk, dv))

    def tokens(n):
        unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
        return (unit(rand(n, H, dk)).to(dt), unit(rand(n, H, dk)).to(dt), (rand(n, H, dv) / 8).to(dt),
                0.9 + 0.1 * torch.rand((n, H), generator=g, device="cuda"),
                torch.rand((n, H), generator=g, device="cuda"))

    def step(b, t, tok):
        q, k, v, al, be = tok
        o = np.zeros((H, dv))
        for h in range(H):
            oo, S[b, h], _ = ref.delta_rule(q[t:t + 1, h], k[t:t + 1, h], v[t:t + 1, h], al[t:t + 1, h], be[t:t + 1, h], S[b, h])
            o[h] = oo[0]
        return o

    def near(x, y):
        assert np.linalg.norm(x - y) <= tol * np.linalg.norm(y)

    def prompts(lens, seqs, has):
        starts = np.concatenate([[0], np.cumsum(lens)])
        tok, N = tokens(int(starts[-1])), int(starts[-1])
        tok = tuple(torch.cat([x, x[:3]]) for x in tok)          # rows behind the last prompt
        o, z = torch.full((N + 3, H, dv), 5.0, device="cuda", dtype=dt), rand(N + 3, H, dv).to(dt)
        p = Prompts(lay, *tok, o, ints(*starts.tolist()), ints(*seqs), ints(*has), norm=norm, norm_gate=z)
        assert lay.prefill(p) == 0
        want = np.zeros((N, H, dv))
        t64 = [f64(x) for x in tok]
        for i, b in enumerate(seqs):
            if not has[i]:
                S[b] = 0
            for t in range(starts[i], starts[i + 1]):
                want[t] = step(b, t, t64)
        near(f64(o[:N]), ref.group_norm(want, f64(norm.weight), None, f64(z[:N]), 1e-5, "silu", False, False))
        assert (o[N:] == 5).all()

    def window():
        for w in range(W):
            st = lay.new_step()
            tok = tokens(B)
            for dst, src in zip((st.q, st.k, st.v, st.gate, st.beta), tok):
                dst.copy_(src)
            assert lay.read(st) == 0 and lay.flush(st) == 0
            z = rand(B, H, dv).to(dt)
            assert lay.normalise(st.o, norm, z) == 0
            t64 = [f64(x) for x in tok]
            want = np.stack([step(b, b, t64) for b in range(B)])
        # the flush's output is exact, and head 1 reads a copy of its state
        near(f64(st.o), ref.group_norm(want, f64(norm.weight), None, f64(z), 1e-5, "silu", False, False))

    prompts([70, 33, 5, 129], [2, 0, 3, 1], [0, 0, 0, 0])
    window()
    cache = StateCache(lay, 3, 8)
    assert lay.save_state(cache, ints(1, 2), ints(2, 0)) == 0
    assert lay.load_state(cache, ints(3, 2), ints(2, 0)) == 0                # fork 1 into 3, requantise 2
    for b, slot in ((3, 2), (2, 0)):
        src = S[1] if b == 3 else S[2]
        got = ref.dequantise(cache.codes[slot].cpu().numpy().astype(np.int64), cache.scale[slot].cpu().numpy())
        # half a code's step of each block, and the state's own roundings
        step_ = np.repeat(f64(cache.scale[slot]), 32, -1)
        assert (np.abs(got - src) <= 0.51 * step_ + 1e-5 * np.abs(src).max()).all()
        S[b] = got
    window()
    prompts([3, 80], [3, 0], [1, 1])
    window()
    near(f64(lay.S), S)
    assert lay.error_word() == 0
