"""The scan's results in every form that a batch may take (tests/test_scan_dispatch.py
holds the batches to their forms): prompts on both sides of the border between two
launches, more prompts than a wave has lanes, segments of several sizes and joins, and
what is refused in them."""
import numpy as np
import pytest
import torch

from tests import sequence_ref as ref
from tests.scan_dispatch_cases import CASES
from tests.test_gpu_scan import COUNT, SEQ, check, f64, ints, make_layer, make_tokens, outside, starts

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.serving import ScanPrompts


def spread(n, B):
    """n sequences of B in another order, and every other one carried on."""
    step = next(s for s in (7, 5, 3, 11, 13) if B % s)
    return [(step * i + 2) % B for i in range(n)], [1 - i % 2 for i in range(n)]


@pytest.mark.parametrize("name", sorted(CASES))
def test_results(name):
    H, G, dk, dv, act, lens, _ = CASES[name]
    n, long = len(lens), max(lens) > 1000
    lay = make_layer(n + 1, H, G, dk, dv, act, seed=800, ranks=[2] * H if H > 20 else None)
    # (slow decays where there are segments: every one of them counts in the last outputs)
    tok = make_tokens(sum(lens) + 3, H, G, dk, dv, act, seed=801, slow=long, packed=True)
    if long:
        lay.A.fill_(0.0)
    S0 = f64(lay.S)
    seqs, has = spread(n, n + 1)
    assert lay.scan(ScanPrompts(lay, *tok, ints(starts(lens, 1)), ints(seqs), ints(has))) == 0
    check(lay, tok, lens, seqs, has, S0, gap=1)


@pytest.mark.parametrize("name", ["both", "both_many", "segments_many", "segments_256_joined", "step_segments_many"])
def test_refused(name):
    """Prompts whose ring holds entries, whose sequence is outside the batch or listed before,
    on both sides of 24 tokens; lists that fall."""
    H, G, dk, dv, act, lens, _ = CASES[name]
    n, B = len(lens), len(lens) + 1
    at = starts(lens)

    def call(seq_start, seqs, count=()):
        lay = make_layer(B, H, G, dk, dv, act, seed=810)
        tok = make_tokens(sum(lens), H, G, dk, dv, act, seed=811)
        for b in count:
            lay.count[b] = 1
        S0 = lay.S.clone()
        assert lay.scan(ScanPrompts(lay, *tok, ints(seq_start), ints(seqs))) == 0
        changed = {b for b in range(B) if not torch.equal(lay.S[b], S0[b])}
        written = {i for i in range(n) if lens[i] and not bool((tok[4][at[i]:at[i + 1]] == 5).any())}
        kept = {i for i in range(n) if lens[i] and bool((tok[4][at[i]:at[i + 1]] == 5).all())}
        return lay.error_word(), changed, written, kept

    full = {i for i in range(n) if lens[i]}
    short, long = min(full, key=lambda i: lens[i]), max(full, key=lambda i: lens[i])
    seqs = list(range(1, n + 1))
    out = {short, long}
    want = lambda err: (err, {i + 1 for i in full - out}, full - out, out)  # noqa: E731
    assert call(at, seqs, count=[short + 1, long + 1]) == want(COUNT)
    bad = list(seqs)
    bad[short], bad[long] = B, -1
    assert call(at, bad) == want(SEQ)
    # a sequence twice: the later prompt is refused
    a, b = sorted((short, long))
    bad = list(seqs)
    bad[b] = bad[a]
    out = {b}
    err, changed, written, kept = call(at, bad)
    assert (err, written, kept) == (SEQ, full - out, out) and changed == {i + 1 for i in full - out}
    fall = list(at)
    fall[n // 2] = at[-1]
    fall[n // 2 + 1] = 0
    assert call(fall, seqs) == (SEQ, set(), set(), full)
    assert call(at[:-1] + [at[-1] + 1], seqs) == (SEQ, set(), set(), full)


def general(q, k, v, dt, rate, S):
    """One head in 64 bits on the device: q, k [T, dk], v [T, dv], dt [T]."""
    o, C = torch.empty_like(v), 1000
    for t in range(0, len(v), C):
        Q, K, V = q[t:t + C], k[t:t + C], v[t:t + C] * dt[t:t + C, None]
        L = torch.cumsum(dt[t:t + C] * rate, 0)
        D = torch.exp((L[None, :] - L[:, None]).clamp(max=0)).tril()
        o[t:t + C] = torch.exp(-L)[:, None] * (Q @ S) + (Q @ K.T.contiguous() * D) @ V
        S = torch.exp(-L[-1]) * S + (K * torch.exp(L - L[-1])[:, None]).T.contiguous() @ V
    return o, S


@pytest.mark.parametrize("H,G,dk,dv,T", [(16, 16, 64, 64, 20000), (16, 16, 128, 64, 17501), (8, 8, 128, 128, 34001)])
def test_long_segments(H, G, dk, dv, T):
    """Segments of 2048 tokens, 32 chunks each.  Roundings of either sign, two a chunk and one a token at most,
    of which those count that have not faded: in quadrature under 2^-24 sqrt(2 T) of the state, twice that allowed; an output is
    rounded to bf16 besides, 2^-8 of itself at most."""
    assert (T >> 10) * G > 256 >= (T >> 11) * G  # (the plan's rule: segments of 2048 tokens)
    lay = make_layer(1, H, G, dk, dv, "bf16", seed=820)
    q, k, v, d, o = make_tokens(T, H, G, dk, dv, "bf16", seed=821, slow=True)
    lay.A.fill_(-1.0)
    S0 = lay.S[0].double()
    assert lay.scan(ScanPrompts(lay, q, k, v, d, o, ints([0, T]))) == 0
    bound = 2.0 ** -23 * (2 * T) ** 0.5
    for h in (0, H - 1):
        oo, S = general(q[:, h].double(), k[:, h].double(), v[:, h].double(), d[:, h].double(), float(torch.exp(lay.A[h].double())), S0[h])
        assert float((lay.S[0, h].double() - S).norm() / S.norm()) <= bound
        e = (o[:, h].double() - oo).abs()
        assert float((e - 2.0 ** -8 * oo.abs()).clamp(min=0).norm() / oo.norm()) <= bound
    assert lay.error_word() == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "dt", "S"])
@pytest.mark.parametrize("H,G,dk,dv,T,act,at", [(4, 2, 128, 64, 1300, "bf16", 83), (4, 2, 128, 64, 1300, "bf16", 700), (32, 32, 64, 64, 1100, "bf16", 300),
                                                (4, 2, 64, 64, 1300, "f32", 450), (3, 3, 16, 32, 1300, "bf16", 83)])
def test_non_finite_values_in_segments(H, G, dk, dv, T, act, at, where, value):
    """A value in one of the first segments reaches no earlier token, and every later one that the recurrence brings it to."""
    if where == "dt" and value < 0:
        value = 3e38                             # (dt is 0 or more: the largest step instead)
    lay = make_layer(1, H, G, dk, dv, act, seed=830, ranks=[2] * H)
    lay.A.fill_(0.0)
    tok = make_tokens(T, H, G, dk, dv, act, seed=831, slow=True)
    if where == "S":
        lay.S[0, 1, 5, 7] = value
    else:
        x = tok[("q", "k", "v", "dt").index(where)]
        x[(at, 1) if where == "dt" else (at, 1, 9)] = value
    S0 = f64(lay.S)
    assert lay.scan(ScanPrompts(lay, *tok, ints([0, T]))) == 0
    o, S = f64(tok[4]), f64(lay.S[0])
    with np.errstate(all="ignore"):
        oo, SS, otol, stol = ref.scan(*(f64(x) for x in tok[:4]), f64(lay.A), S0[0])
    big = 1e30                                   # (3e38 itself leaves sums at the type's end)
    fine, good = np.abs(oo) < big, np.abs(SS) < big
    assert np.isfinite(o[fine]).all() and np.isfinite(S[good]).all()
    assert not np.isfinite(o[~np.isfinite(oo)]).any() and not np.isfinite(S[~np.isfinite(SS)]).any()
    assert outside(o[fine], oo[fine], (ref.HALF[act] * np.abs(oo) + 1.01 * otol)[fine]) == 0
    assert outside(S[good], SS[good], stol[good]) == 0
