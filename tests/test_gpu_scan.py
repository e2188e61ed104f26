"""Prompts through the selective state space scan against the token recurrence in
64 bits.  Tolerances: tests/sequence_ref.py derives what fp32 sums may be off; an
output or a sketch row is rounded once more to its type."""
import numpy as np
import pytest
import torch

from tests import sequence_ref as ref

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.layer import DecodeLayer, TORCH_DTYPE
    from ssm_decode_amd.serving import ScanPrompts

COUNT, SEQ = 1, 4


def f64(x):
    return x.double().cpu().numpy()


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def make_layer(B, H, G, dk, dv, act, seed=0, ranks=None, W=4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = ranks or [min(dk, 1 + (3 * h) % 16) for h in range(H)]
    lay = DecodeLayer("mamba2", B, H, G, dk, dv, W, act, act, np.concatenate([[0], np.cumsum(r)]))
    lay.Pt.copy_(torch.randn(lay.Pt.shape, generator=g, device="cuda") / dk ** 0.5)
    lay.Cmap.copy_(lay.Pt)
    lay.S.copy_(torch.randn(lay.S.shape, generator=g, device="cuda"))
    lay.A.copy_(torch.log(1 + 15 * torch.rand(H, generator=g, device="cuda")))
    lay.U.fill_(7.0)
    return lay


def make_tokens(N, H, G, dk, dv, act, seed=0, slow=False, packed=False):
    """q, k, v, dt, o; slow: decays near 1, so that a prompt's whole past counts."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    d = TORCH_DTYPE[act]
    q, k, v = (rand(N, G, dk) / dk ** 0.5).to(d), (rand(N, G, dk) / dk ** 0.5).to(d), rand(N, H, dv).to(d)
    if packed:
        rows = torch.cat([v.flatten(1), k.flatten(1), q.flatten(1), torch.full((N, 8), 9.0, device="cuda", dtype=d)], 1)
        a, b = H * dv, H * dv + G * dk
        v, k, q = rows[:, :a].unflatten(1, (H, dv)), rows[:, a:b].unflatten(1, (G, dk)), rows[:, b:b + G * dk].unflatten(1, (G, dk))
    u = torch.rand((N, H), generator=g, device="cuda")
    dt = (torch.exp(-7 - 3 * u) if slow else torch.exp(-7 + 5 * u)).to(d)
    return q, k, v, dt, torch.full((N, H, dv), 5.0, device="cuda", dtype=d)


def starts(lens, gap=0):
    return [gap + sum(lens[:i]) for i in range(len(lens) + 1)]


def outside(x, y, tol):
    return int((~(np.abs(x - y) <= tol)).sum())


def check(lay, tok, lens, seqs, has, S0, gap=0, prime=True):
    """All outputs, states and sketches of a call that was made."""
    q, k, v, dt, o = (f64(x) for x in tok)
    at, half = starts(lens, gap), ref.HALF[lay.act]
    S, U, P, off = f64(lay.S), f64(lay.U), f64(lay.Pt), lay.offsets_host
    A = f64(lay.A)
    for i, b in enumerate(seqs):
        s = slice(at[i], at[i + 1])
        oo, SS, otol, stol = ref.scan(q[s], k[s], v[s], dt[s], A, S0[b] if has[i] else 0 * S0[b])
        assert outside(o[s], oo, half * np.abs(oo) + 1.01 * otol) == 0, ("o", i)
        assert outside(S[b], SS, stol) == 0, ("S", i)
        if prime:
            # (of the fp32 state that was written)
            uu, utol = ref.sketch(S[b], P, off)
            assert outside(U[b], uu, half * np.abs(uu) + 1.01 * utol) == 0, ("U", i)
            for n, h in enumerate(lay.dense_heads):
                assert outside(f64(lay.Scopy[b, n]), S[b, h], half * np.abs(S[b, h])) == 0
    for b in set(range(lay.B)) - set(seqs):
        assert (S[b] == S0[b]).all() and (U[b] == 7).all()
    if not prime:
        assert (U == 7).all()
    assert (o[:at[0]] == 5).all() and (o[at[-1]:] == 5).all()
    assert lay.error_word() == 0


LENS = {"short": [3, 1, 0, 17, 2], "ragged": [64, 1, 0, 65, 63, 130, 24, 25], "long": [700], "many": [200, 5, 300, 129]}


@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,H,G", [(16, 32, 3, 3), (64, 64, 6, 2), (128, 64, 16, 1), (128, 64, 4, 4), (128, 128, 5, 1),
                                       (128, 64, 22, 2), (64, 64, 11, 1)])
def test_prompts(dk, dv, H, G, act, lens):
    lens = LENS[lens]
    n = len(lens)
    lay = make_layer(n + 2, H, G, dk, dv, act, seed=dk + H, ranks=[0] + [min(dk, 1 + 3 * h % 16) for h in range(1, H)])
    tok = make_tokens(sum(lens) + 5, H, G, dk, dv, act, seed=3, packed=H % 2 == 0)
    S0 = f64(lay.S)
    seqs, has = [(3 * i + 1) % (n + 2) if (n + 2) % 3 else n + 1 - i for i in range(n)], [i % 2 for i in range(n)]
    assert lay.scan(ScanPrompts(lay, *tok, ints(starts(lens, 2)), ints(seqs), ints(has))) == 0
    check(lay, tok, lens, seqs, has, S0, gap=2)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("prime", [True, False])
def test_a_long_memory(act, prime):
    """Decays near 1: every token of a prompt of several segments counts in its last outputs."""
    lens = [1500, 90]
    lay = make_layer(2, 4, 2, 128, 64, act, seed=9)
    tok = make_tokens(sum(lens), 4, 2, 128, 64, act, seed=10, slow=True)
    S0 = f64(lay.S)
    assert lay.scan(ScanPrompts(lay, *tok, ints(starts(lens)), prime=prime)) == 0
    check(lay, tok, lens, [0, 1], [1, 1], S0, prime=prime)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_steps_of_any_size(act):
    """dt of zero (nothing happens but an output) and so large that all is forgotten."""
    lens = [150]
    lay = make_layer(1, 4, 1, 128, 64, act, seed=19)
    tok = make_tokens(150, 4, 1, 128, 64, act, seed=20)
    tok[3][::3] = 0
    tok[3][5::17] = 40.0
    tok[3][40:48] = 3e4
    S0 = f64(lay.S)
    assert lay.scan(ScanPrompts(lay, *tok, ints(starts(lens)))) == 0
    check(lay, tok, lens, [0], [1], S0)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_small_difference_of_large_terms(act):
    """The second token takes back what the first wrote, to one part in 2^12: the outputs after it are
    what every bit of the state's operands leaves."""
    T, H, dk, dv = 130, 2, 128, 64
    lay = make_layer(1, H, 1, dk, dv, act, seed=29)
    q, k, v, dt, o = make_tokens(T, H, 1, dk, dv, act, seed=30, slow=True)
    lay.S.zero_()
    dt.fill_(0)
    dt[0], dt[1] = 0.5, 0.5
    k[1] = k[0]
    v[1] = -v[0]
    lay.A.fill_(-20.0)                   # decays of 1 - 1e-9: one in fp32
    lay.S.copy_(2.0 ** -12 * torch.randn(lay.S.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)))
    S0 = f64(lay.S)
    assert lay.scan(ScanPrompts(lay, q, k, v, dt, o, ints([0, T]))) == 0
    check(lay, (q, k, v, dt, o), [T], [0], [1], S0)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 90, 1300])
def test_empty_and_repeated_calls(act, T):
    """A prompt in two calls is the prompt in one, to the bounds; an empty prompt leaves or clears its state."""
    lay = make_layer(3, 4, 2, 64, 64, act, seed=39)
    tok = make_tokens(T, 4, 2, 64, 64, act, seed=40)
    S0 = f64(lay.S)
    cut = T // 2 + 1
    for a, b in ((0, cut), (cut, T)):
        assert lay.scan(ScanPrompts(lay, *tok, ints([a, b, b, b]), ints([1, 0, 2]), ints([1, 1, 0]))) == 0
    check(lay, tuple(torch.cat([x, x[:0]]) for x in tok), [T, 0, 0], [1, 0, 2], [1, 1, 0], S0)


# ------------------------------------------------- infinities and NaN
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "dt", "S"])
def test_non_finite_values_reach_no_earlier_token(where, value, act):
    if where == "dt" and value < 0:
        pytest.skip("dt is 0 or more")
    T, H, G, dk, dv, at = 200, 4, 2, 128, 64, 83
    lay = make_layer(1, H, G, dk, dv, act, seed=49)
    tok = make_tokens(T, H, G, dk, dv, act, seed=50, slow=True)
    if where == "S":
        lay.S[0, 1, 5, 7] = value
    else:
        x = tok[("q", "k", "v", "dt").index(where)]
        x[(at, 1) if where == "dt" else (at, 1 if where == "v" else 0, 9)] = value
    S0 = f64(lay.S)
    assert lay.scan(ScanPrompts(lay, *tok, ints([0, T]))) == 0
    o, S = f64(tok[4]), f64(lay.S[0])
    with np.errstate(all="ignore"):
        oo, SS, otol, stol = ref.scan(*(f64(x) for x in tok[:4]), f64(lay.A), S0[0])
    assert (np.isfinite(o) == np.isfinite(oo)).all() and (np.isfinite(S) == np.isfinite(SS)).all()
    ok = np.isfinite(oo) & np.isfinite(otol)
    assert outside(o[ok], oo[ok], (ref.HALF[act] * np.abs(oo) + 1.01 * otol)[ok]) == 0
    ok = np.isfinite(SS) & np.isfinite(stol)
    assert outside(S[ok], SS[ok], stol[ok]) == 0


# --------------------------------------------------------- refused prompts
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[3, 2, 4], [300, 70, 129]])
def test_refused_prompts(lens, act):
    N = sum(lens)

    def call(seq_start, seqs, count=None):
        lay = make_layer(4, 3, 1, 64, 64, act, seed=59)
        tok = make_tokens(N, 3, 1, 64, 64, act, seed=60)
        if count is not None:
            lay.count[count] = 1
        S0 = lay.S.clone()
        assert lay.scan(ScanPrompts(lay, *tok, ints(seq_start), ints(seqs))) == 0
        same = [bool(torch.equal(lay.S[b], S0[b])) for b in range(4)]
        kept = [bool((tok[4][a:b] == 5).all()) for a, b in zip(starts(lens), starts(lens)[1:])]
        return lay.error_word(), same, kept

    s = starts(lens)
    assert call(s, [0, 1, 2], count=1) == (COUNT, [False, True, False, True], [False, True, False])
    assert call(s, [0, 4, 2]) == (SEQ, [False, True, False, True], [False, True, False])
    assert call(s, [0, -1, 2]) == (SEQ, [False, True, False, True], [False, True, False])
    assert call(s, [1, 2, 1]) == (SEQ, [True, False, False, True], [False, False, True])
    assert call([s[0], s[2], s[1], s[3]], [0, 1, 2]) == (SEQ, [True] * 4, [True] * 3)
    assert call([s[0], s[1], s[2], s[3] + 1], [0, 1, 2]) == (SEQ, [True] * 4, [True] * 3)
    assert call([-1, s[1], s[2], s[3]], [0, 1, 2]) == (SEQ, [True] * 4, [True] * 3)
    assert call([N + 900] * 4, [0, 1, 2]) == (SEQ, [True] * 4, [True] * 3)
    # prompts far past the end, and of negative length: nothing of their segments is read
    assert call([0, 1 << 30, 1 << 30, 1 << 30], [0, 1, 2]) == (SEQ, [True] * 4, [True] * 3)
    assert call([0, 2 ** 31 - 1, 0, 2 ** 31 - 1], [0, 1, 2]) == (SEQ, [True] * 4, [True] * 3)
    assert call([1 << 20, 0, 1 << 20, 0], [0, 1, 2]) == (SEQ, [True] * 4, [True] * 3)


# ------------------------------------------------ streams, graphs, offsets
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_captured_and_replayed_with_other_lists(act):
    lens = [[300, 20, 129], [7, 400, 42]]
    lay = make_layer(3, 4, 2, 128, 64, act, seed=69)
    tok = make_tokens(449, 4, 2, 128, 64, act, seed=70)
    st, has = ints(starts(lens[0])), ints([0, 0, 0])
    pr = ScanPrompts(lay, *tok, st, has_state=has)
    S0 = f64(lay.S)
    lay.scan(pr)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert lay.scan(pr) == 0
    for n in (1, 0, 1):
        st.copy_(ints(starts(lens[n])))
        tok[4].fill_(5.0)
        lay.U.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check(lay, tok, lens[n], [0, 1, 2], [0, 0, 0], S0)


def test_two_calls_at_once():
    lens = [513, 64]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    made = []
    for n in range(2):
        lay = make_layer(2, 4, 1, 128, 64, "bf16", seed=79 + n)
        tok = make_tokens(577, 4, 1, 128, 64, "bf16", seed=80 + n)
        made.append((lay, tok, f64(lay.S), ScanPrompts(lay, *tok, ints(starts(lens)))))
    torch.cuda.synchronize()
    for s in side:
        with torch.cuda.stream(s):
            torch.cuda._sleep(1 << 24)
    for s, m in zip(side, made):
        assert m[0].scan(m[3], stream=s.cuda_stream) == 0
    torch.cuda.synchronize()
    for lay, tok, S0, _ in made:
        check(lay, tok, lens, [0, 1], [1, 1], S0)


def test_rows_far_apart():
    """Offsets past 2^32 bytes within a prompt."""
    T, H, dk, dv = 70, 1, 64, 64
    lay = make_layer(1, H, 1, dk, dv, "bf16", seed=89)
    tok = list(make_tokens(T, H, 1, dk, dv, "bf16", seed=90))
    wide = 1 << 25
    far = torch.empty(wide * (T - 1) + 512, dtype=torch.bfloat16, device="cuda")
    for n, at in ((0, 0), (1, 64), (2, 128), (4, 192)):
        view = far.as_strided((T, 1, 64), (wide, 64, 1), at)
        view.copy_(tok[n])
        tok[n] = view
    S0 = f64(lay.S)
    assert lay.scan(ScanPrompts(lay, *tok, ints([0, T]))) == 0
    check(lay, tuple(tok), [T], [0], [1], S0)


def test_prompts_are_the_decode_steps_start():
    """A prompt, then decode steps: the read's exact part and the flush go on from the scan's state and sketch."""
    B, H, G, dk, dv, W = 2, 4, 2, 64, 64, 4
    lay = make_layer(B, H, G, dk, dv, "f32", seed=99, W=W)
    tok = make_tokens(2 * 90, H, G, dk, dv, "f32", seed=100)
    S0 = f64(lay.S)
    assert lay.scan(ScanPrompts(lay, *tok, ints([0, 90, 180]))) == 0
    more = make_tokens(W * B, H, G, dk, dv, "f32", seed=101)
    for w in range(W):
        st = lay.new_step()
        for dst, src in zip((st.q, st.k, st.v, st.gate), more):
            dst.copy_(src[w * B:(w + 1) * B])
        assert lay.read(st) == 0 and lay.flush(st) == 0
    for b in range(B):
        one = [np.concatenate([f64(x)[90 * b:90 * b + 90], f64(y)[b::B]]) for x, y in zip(tok[:4], more[:4])]
        o, S, otol, stol = ref.scan(*one, f64(lay.A), S0[b])
        # (the decode path's decays are exponentials of rounded products: 2^-20 of a logarithm up to 16)
        assert outside(f64(lay.S[b]), S, stol + 2.0 ** -16 * np.abs(S).max()) == 0
        assert outside(f64(st.o[b]), o[-1], otol[-1] + 2.0 ** -14 * np.abs(o).max()) == 0
    assert lay.error_word() == 0
