"""Prompts of the gated delta rule on the GPU against the token recurrence in
64 bits: shapes, types, lengths, strides, lists, refusals, graphs, and the
decode steps that go on from a prompt."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd import abi
    from ssm_decode_amd.layer import DecodeLayer, TORCH_DTYPE
    from ssm_decode_amd.serving import Prompts

SENTINEL = 777.0
EPS32 = 2.0 ** -24


def make_layer(B, H, dk, dv, act, ranks=None, seed=0, W=4):
    ranks = [(2 + 3 * h) % 9 for h in range(H)] if ranks is None else ranks
    off = np.concatenate([[0], np.cumsum(ranks)]).astype(np.int32)
    lay = DecodeLayer("gdn", B, H, H, dk, dv, W, act, act, off)
    g = torch.Generator(device="cuda").manual_seed(seed)
    lay.S.copy_(0.1 * torch.randn(lay.S.shape, generator=g, device="cuda"))
    lay.Pt.copy_(torch.randn(lay.Pt.shape, generator=g, device="cuda") / dk ** 0.5)
    lay.Cmap.copy_(lay.Pt)
    return lay


def make_tokens(N, H, dk, dv, act, seed=0, packed=False, alpha=None, pad=0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    dt = TORCH_DTYPE[act]
    q = torch.nn.functional.normalize(torch.randn((N, H, dk), generator=g, device="cuda"), dim=-1).to(dt)
    k = torch.nn.functional.normalize(torch.randn((N, H, dk), generator=g, device="cuda"), dim=-1).to(dt)
    v = (torch.randn((N, H, dv), generator=g, device="cuda") / dv ** 0.5).to(dt)
    if packed:                    # slices of one projection's rows, with a gap behind them
        rows = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1),
                          torch.zeros((N, 16), device="cuda", dtype=dt)], 1)
        q, k, v = (rows[:, a:a + H * d].unflatten(1, (H, d)) for a, d in ((0, dk), (H * dk, dk), (2 * H * dk, dv)))
    al = 0.9 + 0.1 * torch.rand((N, H), generator=g, device="cuda") if alpha is None else alpha
    be = torch.rand((N, 2 * H + 1), generator=g, device="cuda")[:, :H] if packed else \
        torch.rand((N, H), generator=g, device="cuda")
    o = torch.full((N + pad, H * dv + (24 if packed else 0)), SENTINEL, device="cuda", dtype=dt)
    o = o[:, :H * dv].unflatten(1, (H, dv))
    return q, k, v, al, be, o


def f64(x):
    return x.double().cpu().numpy()


def expect(lay, S0, tok, lens, starts, seqs, has, skip=()):
    """Reference outputs {token: [H, dv]}, states and the tolerance's scale."""
    q, k, v, al, be, _ = [f64(x) for x in tok]
    S = f64(S0)
    o, top = {}, 0.0
    for i, n in enumerate(lens):
        if i in skip:
            continue
        a, b = starts[i], seqs[i]
        for h in range(lay.H):
            s0 = S[b, h] if has[i] else np.zeros_like(S[b, h])
            oo, S[b, h], m = ref.delta_rule(q[a:a + n, h], k[a:a + n, h], v[a:a + n, h], al[a:a + n, h], be[a:a + n, h], s0)
            top = max(top, m)
            for t in range(n):
                o.setdefault(a + t, np.zeros((lay.H, lay.dv)))[h] = oo[t]
    return o, S, top


def check(lay, S0, tok, lens, starts, seqs, has, skip=(), prime=True):
    """The bounds.  Every operation is fp32 with fp32 sums: a token adds at
    most (dk + 8) roundings of 2^-24 of the state's column norm, and the
    transition does not enlarge them for |k| <= 1, 0 <= alpha, beta <= 1; keys
    rounded to bf16 may have norms up to 1 + 2^-8, which a product over the
    tested lengths keeps under 2.  Then one rounding to the output's type, half
    a step of it."""
    o, S, top = expect(lay, S0, tok, lens, starts, seqs, has, skip)
    n = max([x for i, x in enumerate(lens) if i not in skip], default=0)
    slack = 2 * (n + 2) * (lay.dk + 8) * EPS32 * max(top, 1e-30)
    half = torch.finfo(TORCH_DTYPE[lay.act]).eps / 2
    got_S = f64(lay.S)
    assert np.isfinite(got_S).all()
    assert np.abs(got_S - S).max() <= slack + EPS32 * np.abs(S).max()
    got = f64(tok[5])
    for t in range(len(got)):
        if t in o:
            assert (np.abs(got[t] - o[t]) <= half * np.abs(o[t]) * (1 + slack) + slack).all(), t
        else:
            assert (got[t] == float(torch.tensor(SENTINEL).to(tok[5].dtype))).all(), t
    # the errors of many roundings do not line up: the norm is far nearer than the
    # bound (random signs over dk terms and the few tokens that a decay keeps)
    den = np.linalg.norm(S)
    if den:
        assert np.linalg.norm(got_S - S) <= 8 * lay.dk ** 0.5 * EPS32 * den
    if prime:
        P, off = f64(lay.Pt), lay.offsets_host
        dense = {h: j for j, h in enumerate(lay.dense_heads)}
        for i in range(len(lens)):
            if i in skip:
                continue
            b = seqs[i]
            for h in range(lay.H):
                if h in dense:
                    assert torch.equal(lay.Scopy[b, dense[h]], lay.S[b, h].to(lay.Scopy.dtype))
                    continue
                r = slice(off[h], off[h + 1])
                U = P[r] @ got_S[b, h]
                lim = half * np.abs(U) + (lay.dk + 2) * EPS32 * (np.abs(P[r]) @ np.abs(got_S[b, h]))
                assert (np.abs(f64(lay.U[b, r]) - U) <= lim * (1 + half)).all()


def run(lay, tok, lens, starts=None, seqs=None, has=None, prime=True, expect_rc=0):
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if starts is None:
        starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    N = len(tok[0])
    p = Prompts(lay, *tok[:5], tok[5][:N], dev(starts), dev(seqs), dev(has), prime)
    assert lay.prefill(p) == expect_rc
    torch.cuda.synchronize()
    return p, starts


SHAPES = [(16, 32), (64, 64), (128, 64), (128, 128)]
LENS = [[1], [2], [0], [5, 0, 1], [16, 17, 15], [33, 1, 64, 20], [63, 64, 65], [127, 129], [200, 3, 70]]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
def test_prompts(act, dk, dv, lens):
    H, n = 3, len(lens)
    B = n + 2
    lay = make_layer(B, H, dk, dv, act, seed=sum(lens))
    tok = make_tokens(sum(lens), H, dk, dv, act, seed=dk + dv, packed=True, pad=3)
    S0 = lay.S.clone()
    seqs = [(2 * i + 1) % B for i in range(n)] if B % 2 else [B - 1 - i for i in range(n)]
    has = [i % 2 for i in range(n)]
    _, starts = run(lay, tok, lens, seqs=seqs, has=has)
    assert lay.error_word() == 0
    check(lay, S0, tok, lens, starts, seqs, has)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_long_prompt_from_its_state(act):
    lay = make_layer(2, 2, 128, 128, act, seed=5)
    tok = make_tokens(700, 2, 128, 128, act, seed=6)
    S0 = lay.S.clone()
    _, starts = run(lay, tok, [700])
    check(lay, S0, tok, [700], starts, [0], [1])


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["zeros", "ones", "tiny", "mixed", "one-zero"])
def test_decays_at_the_ends_of_their_range(act, kind):
    """Decays of zero, one and down to 2^-126: ratios of their products would
    overflow or divide by zero."""
    N, H = 150, 2
    lay = make_layer(2, H, 64, 64, act, seed=7)
    al = {"zeros": torch.zeros(N, H), "ones": torch.ones(N, H), "tiny": torch.full((N, H), 2.0 ** -126),
          "mixed": torch.rand(N, H).pow(20), "one-zero": torch.ones(N, H)}[kind].clone()
    if kind == "one-zero":
        al[77] = 0
    tok = make_tokens(N, H, 64, 64, act, seed=8, alpha=al.cuda())
    S0 = lay.S.clone()
    _, starts = run(lay, tok, [N], seqs=[1])
    check(lay, S0, tok, [N], starts, [1], [1])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_repeated_keys_and_large_values(act):
    """The same key at every token with beta near one (the triangular system's
    worst case), and values and states far from one."""
    N, H = 130, 2
    for scale in (1.0, 2.0 ** 60, 2.0 ** -60):
        lay = make_layer(1, H, 64, 64, act, seed=9)
        lay.S.mul_(scale)
        q, k, v, al, be, o = make_tokens(N, H, 64, 64, act, seed=10)
        k.copy_(k[:1].expand_as(k))
        be.copy_(1.0 - be * 2.0 ** -6)
        v.mul_(scale)
        tok = (q, k, v, al, be, o)
        S0 = lay.S.clone()
        _, starts = run(lay, tok, [N])
        check(lay, S0, tok, [N], starts, [0], [1])


def test_matches_the_decode_step_bit_for_bit_in_f32_single_tokens():
    """A single token through the prompt path and sketchssm_full_step compute
    the same numbers within an fp32 rounding."""
    lay = make_layer(3, 4, 64, 64, "f32", seed=11)
    other = make_layer(3, 4, 64, 64, "f32", seed=11)
    tok = make_tokens(3, 4, 64, 64, "f32", seed=12)
    run(lay, tok, [1, 1, 1])
    st = other.new_step()
    for dst, src in zip((st.q, st.k, st.v, st.gate, st.beta), tok):
        dst.copy_(src)
    assert other.full_step(st) == 0
    torch.cuda.synchronize()
    torch.testing.assert_close(lay.S, other.S, rtol=1e-5, atol=1e-6)
    torch.testing.assert_close(tok[5], st.o, rtol=1e-5, atol=1e-6)


def test_refused_entries_leave_everything_else():
    """Sequences out of range, listed twice, with buffered entries, and bad
    ranges are reported and skipped; the others are done."""
    H, dk, dv = 2, 64, 64
    for act in ("bf16", "f32"):
        for lens in ([70, 70, 70, 70, 70], [3, 3, 3, 3, 3]):
            N = sum(lens)
            lay = make_layer(5, H, dk, dv, act, seed=13)
            lay.count[3] = 1
            tok = make_tokens(N, H, dk, dv, act, seed=14)
            S0, U0 = lay.S.clone(), lay.U.clone()
            seqs = [4, -1, 4, 3, 0]
            _, starts = run(lay, tok, lens, seqs=seqs)
            assert lay.error_word() == abi.SKSSM_ERRBIT_SEQ | abi.SKSSM_ERRBIT_COUNT
            check(lay, S0, tok, lens, starts, seqs, [1] * 5, skip=(1, 2, 3))
            assert torch.equal(lay.S[1:4], S0[1:4]) and torch.equal(lay.U[1:4], U0[1:4])
            assert lay.count[3].tolist() == [1] * H


@pytest.mark.parametrize("starts", [
    [100, 30, 60, 200], [0, 70, 60, 200], [-5, 70, 140, 200], [0, 70, 140, 999], [0, 2000000000, 140, 200],
    [-2147483648, 2147483647, 140, 200], [0, 70, 140, 60], [0, 5, 3, 9], [0, 3, 9, 201], [300, 300, 300, 300]])
@pytest.mark.parametrize("tokens", [200, 150, 12])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_bad_list_of_tokens_is_refused_whole(starts, tokens, act):
    lay = make_layer(3, 2, 64, 64, act, seed=15)
    tok = make_tokens(tokens, 2, 64, 64, act, seed=16)
    S0, U0 = lay.S.clone(), lay.U.clone()
    run(lay, tok, None, starts=starts)
    assert lay.error_word() == abi.SKSSM_ERRBIT_SEQ
    assert torch.equal(lay.S, S0) and torch.equal(lay.U, U0) and (tok[5].float() == torch.tensor(SENTINEL).to(tok[5].dtype).float()).all()


@pytest.mark.parametrize("starts", [[0, 100, 100, 100], [50, 60, 150, 170], [0, 0, 0, 200], [200, 200, 200, 200]])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_lists_that_leave_tokens_out(starts, act):
    lay = make_layer(3, 2, 64, 64, act, seed=15)
    tok = make_tokens(200, 2, 64, 64, act, seed=16)
    S0 = lay.S.clone()
    run(lay, tok, None, starts=starts)
    assert lay.error_word() == 0
    check(lay, S0, tok, [b - a for a, b in zip(starts, starts[1:])], starts, [0, 1, 2], [1] * 3)


@pytest.mark.parametrize("n,lens", [(70, "mixed"), (70, "long"), (200, "mixed")])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_many_prompts(n, lens, act):
    """More prompts than a wave's lanes, short and long among them."""
    rng = np.random.default_rng(n)
    lens = (rng.choice([0, 1, 3, 16, 17, 40, 64, 130], n) if lens == "mixed" else rng.integers(60, 140, n)).tolist()
    lay = make_layer(n, 2, 64, 64, act, seed=70)
    tok = make_tokens(sum(lens), 2, 64, 64, act, seed=71)
    S0 = lay.S.clone()
    seqs = rng.permutation(n).tolist()
    has = rng.integers(0, 2, n).tolist()
    _, starts = run(lay, tok, lens, seqs=seqs, has=has)
    assert lay.error_word() == 0
    check(lay, S0, tok, lens, starts, seqs, has)


@pytest.mark.parametrize("dk,dv", SHAPES[1:])
@pytest.mark.parametrize("lens", [[4096], [4097], [5000, 0, 7300], [12300, 5, 1], [1024, 1025, 10300], [1, 8200], [2048] * 4 + [12300], [2048], [2049], [511, 512, 513, 6700]],
                         ids=lambda x: "-".join(map(str, x)))
def test_few_long_prompts(dk, dv, lens):
    """Few tiles with many tokens: prompts in segments (of 512 tokens here), the
    first from its state and from zero, prompts of one segment among them."""
    H, n = 1, len(lens)
    lay = make_layer(n + 1, H, dk, dv, "bf16", seed=80, ranks=[5])
    tok = make_tokens(sum(lens), H, dk, dv, "bf16", seed=81, packed=True, pad=2, alpha=None)
    tok[3][:] = 1 - (1 - tok[3]) * 0.01            # slow decays: a segment's start is felt at its end
    S0 = lay.S.clone()
    seqs, has = [n - i for i in range(n)], [(i + 1) % 2 for i in range(n)]
    for rep in range(2):                           # the same workspace twice, from the same states
        lay.S.copy_(S0)
        _, starts = run(lay, tok, lens, seqs=seqs, has=has)
        assert lay.error_word() == 0
        check(lay, S0, tok, lens, starts, seqs, has)


def test_few_long_prompts_refused_and_replayed():
    """A refused prompt among segmented ones, and a captured call."""
    lens = [4500, 4600, 4400]
    N = sum(lens)
    lay = make_layer(3, 1, 64, 64, "bf16", seed=82, ranks=[0])
    tok = make_tokens(N, 1, 64, 64, "bf16", seed=83)
    S0 = lay.S.clone()
    lay.count[2] = 2
    run(lay, tok, lens, seqs=[0, 2, 0])
    assert lay.error_word() == abi.SKSSM_ERRBIT_SEQ | abi.SKSSM_ERRBIT_COUNT
    check(lay, S0, tok, lens, [0, 4500, 9100, 13500], [0, 2, 0], [1] * 3, skip=(1, 2))
    lay.count.zero_()
    pr = Prompts(lay, *tok, torch.tensor([0, 4500, 9100, 13500], dtype=torch.int32, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert lay.prefill(pr) == 0
    for rep in range(3):
        for dst, src in zip(tok, make_tokens(N, 1, 64, 64, "bf16", seed=84 + rep)):
            dst.copy_(src)
        lay.S.copy_(S0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(lay, S0, tok, lens, [0, 4500, 9100, 13500], [0, 1, 2], [1] * 3)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_no_prompts_and_empty_prompts(act):
    lay = make_layer(3, 2, 64, 64, act, seed=17)
    S0 = lay.S.clone()
    tok = make_tokens(0, 2, 64, 64, act)
    run(lay, tok, [])
    assert torch.equal(lay.S, S0)
    run(lay, tok, [0, 0, 0], has=[1, 0, 1])
    assert torch.equal(lay.S[0], S0[0]) and torch.equal(lay.S[2], S0[2]) and not lay.S[1].any()
    check(lay, S0, tok, [0, 0, 0], [0] * 4, [0, 1, 2], [1, 0, 1])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_nan_stays_in_its_own_prompt_and_head(act):
    lay = make_layer(3, 2, 64, 64, act, seed=18)
    lens = [70, 80, 50]
    tok = make_tokens(200, 2, 64, 64, act, seed=19)
    tok[2][75, 1, 5] = float("nan")
    tok[2][76, 0, 7] = float("inf")
    run(lay, tok, lens)
    bad = ~torch.isfinite(lay.S)
    assert not bad[0].any() and not bad[2].any()
    assert bad[1, 1, :, 5].any() and not bad[1, 1, :, :5].any() and not bad[1, 1, :, 6:].any()
    assert bad[1, 0, :, 7].any() and not bad[1, 0, :, :7].any() and not bad[1, 0, :, 8:].any()
    assert torch.isfinite(tok[5].float()[:70]).all() and torch.isfinite(tok[5].float()[150:]).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_zero_state_ignores_what_the_buffer_held(act):
    lay = make_layer(2, 2, 64, 64, act, seed=20)
    lay.S.fill_(float("nan"))
    tok = make_tokens(150, 2, 64, 64, act, seed=21)
    run(lay, tok, [100, 50], has=[0, 0])
    check(lay, torch.zeros_like(lay.S), tok, [100, 50], [0, 100, 150], [0, 1], [0, 0])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_prompt_in_two_parts_equals_it_in_one(act):
    a, b = make_layer(1, 2, 128, 128, act, seed=22), make_layer(1, 2, 128, 128, act, seed=22)
    tok = make_tokens(300, 2, 128, 128, act, seed=23)
    S0 = a.S.clone()
    run(a, tok, [300])
    o = torch.empty_like(tok[5])
    for lo, hi in ((0, 101), (101, 300)):
        part = tuple(x[lo:hi] for x in tok[:5]) + (o[lo:hi],)
        run(b, part, [hi - lo])
    check(b, S0, tok[:5] + (o,), [300], [0, 300], [0], [1])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_long_row_strides(act):
    """Rows so far apart that offsets pass 32 bits."""
    N, H, dk, dv = 70, 2, 64, 64
    stride = 1 << 25                             # 70 rows: over 2^31 elements
    lay = make_layer(1, H, dk, dv, act, seed=24)
    q, k, v, al, be, o = make_tokens(N, H, dk, dv, act, seed=25)
    far = torch.empty(N * stride, device="cuda", dtype=TORCH_DTYPE[act])
    at = lambda i, d: far.as_strided((N, H, d), (stride, d, 1), i * 1024)  # noqa: E731
    tok = []
    for i, (x, d) in enumerate(((q, dk), (k, dk), (v, dv), (o, dv))):
        y = at(i, d)
        y.copy_(x)
        tok.append(y)
    S0 = lay.S.clone()
    tok = (tok[0], tok[1], tok[2], al, be, tok[3])
    _, starts = run(lay, tok, [N])
    check(lay, S0, tok, [N], starts, [0], [1])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_on_another_stream_and_twice_at_once(act):
    """Two layers' prompts on two streams, each with its own workspace."""
    lays = [make_layer(2, 3, 128, 128, act, seed=26 + i) for i in range(2)]
    toks = [make_tokens(400, 3, 128, 128, act, seed=28 + i) for i in range(2)]
    S0 = [x.S.clone() for x in lays]
    start = torch.tensor([0, 150, 400], dtype=torch.int32, device="cuda")
    pr = [Prompts(lay, *tok, start) for lay, tok in zip(lays, toks)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            assert lays[i].prefill(pr[i]) == 0
    torch.cuda.synchronize()
    for i in range(2):
        check(lays[i], S0[i], toks[i], [150, 250], [0, 150, 400], [0, 1], [1, 1])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_same_call_twice_gives_the_same_bits(act):
    lay = make_layer(4, 3, 128, 128, act, seed=30)
    tok = make_tokens(500, 3, 128, 128, act, seed=31)
    S0, outs = lay.S.clone(), []
    for _ in range(2):
        lay.S.copy_(S0)
        run(lay, tok, [130, 1, 300, 69])
        outs.append([x.clone() for x in (lay.S, lay.U, tok[5])])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens", [[3, 9], [100, 90]], ids=["short", "long"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_graph_replays(lens, act):
    """Captured once, replayed with other prompts in the same buffers and eager
    work between the replays."""
    N = sum(lens)
    lay = make_layer(2, 2, 128, 128, act, seed=32)
    tok = make_tokens(N, 2, 128, 128, act, seed=33)
    starts = [0, lens[0], N]
    pr = Prompts(lay, *tok, torch.tensor(starts, dtype=torch.int32, device="cuda"))
    S0 = lay.S.clone()
    lay.prefill(pr)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert lay.prefill(pr) == 0
    for rep in range(4):
        new = make_tokens(N, 2, 128, 128, act, seed=40 + rep)
        for dst, src in zip(tok, new):
            dst.copy_(src)
        lay.S.copy_(S0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(lay, S0, tok, lens, starts, [0, 1], [1, 1])


def test_prompt_then_decode_window():
    """A prompt, then a window of reads and its flush: the flush output and the
    state are those of the recurrence over prompt and decode tokens."""
    B, H, dk, dv, W, N = 3, 2, 64, 64, 4, 90
    lay = make_layer(B, H, dk, dv, "f32", seed=50, W=W, ranks=[8, 0])
    tok = make_tokens(N, H, dk, dv, "f32", seed=51)
    lens = [40, 30, 20]
    S0 = lay.S.clone()
    _, starts = run(lay, tok, lens, has=[0, 0, 1])
    _, S, _ = expect(lay, S0, tok, lens, starts, [0, 1, 2], [0, 0, 1])
    for w in range(W):
        st = lay.new_step()
        dec = make_tokens(B, H, dk, dv, "f32", seed=60 + w)
        for dst, src in zip((st.q, st.k, st.v, st.gate, st.beta), dec):
            dst.copy_(src)
        assert lay.read(st) == 0
        assert lay.flush(st) == 0
        q, k, v, al, be, _ = [f64(x) for x in dec]
        o = np.zeros((B, H, dv))
        for b in range(B):
            for h in range(H):
                oo, S[b, h], _ = ref.delta_rule(q[b:b + 1, h], k[b:b + 1, h], v[b:b + 1, h], al[b:b + 1, h], be[b:b + 1, h], S[b, h])
                o[b, h] = oo[0]
        # a dense-fallback head reads its state's copy (exact in f32) at every step
        got = f64(st.o)
        assert np.linalg.norm(got[:, 1] - o[:, 1]) <= 1e-5 * np.linalg.norm(o[:, 1])
    assert np.linalg.norm(got - o) <= 1e-5 * np.linalg.norm(o)
    assert np.linalg.norm(f64(lay.S) - S) <= 1e-5 * np.linalg.norm(S)
    assert lay.error_word() == 0


@pytest.mark.parametrize("tokens,starts", [(200, [150, 100, 50, 10]), (13000, [13000, 0]), (13000, [14000, 15000]),
                                           (13000, [-2000, 12000]), (13000, [9000, 8000, 12500])])
def test_a_list_that_only_falls_is_reported(tokens, starts):
    """Lists whose prompts no workgroup of the chunks comes to."""
    n = len(starts) - 1
    lay = make_layer(n, 1, 64, 64, "bf16", seed=15, ranks=[4])
    tok = make_tokens(tokens, 1, 64, 64, "bf16", seed=16)
    S0 = lay.S.clone()
    run(lay, tok, None, starts=starts)
    assert lay.error_word() == abi.SKSSM_ERRBIT_SEQ
    assert torch.equal(lay.S, S0) and (tok[5].float() == torch.tensor(SENTINEL).to(tok[5].dtype).float()).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_short_and_long_prompts_together(dk, dv, act):
    """Lengths about those where a prompt changes from one form to the other."""
    lens = [16, 17, 24, 25, 1, 32, 33, 0, 48, 49, 64, 65]
    n = len(lens)
    lay = make_layer(n, 3, dk, dv, act, seed=90)
    tok = make_tokens(sum(lens), 3, dk, dv, act, seed=91, packed=True, pad=1)
    S0 = lay.S.clone()
    seqs, has = list(range(n))[::-1], [i % 3 > 0 for i in range(n)]
    _, starts = run(lay, tok, lens, seqs=seqs, has=[int(x) for x in has])
    assert lay.error_word() == 0
    check(lay, S0, tok, lens, starts, seqs, has)


@pytest.mark.parametrize("act,n", [("bf16", 3), ("bf16", 100), ("f32", 3), ("f32", 100), ("bf16", 9000)])
def test_the_last_of_very_many_states(act, n):
    """States whose offsets pass 32 bits: of 2^17 + 8 sequences of one 128 x 128
    head, the first and the last."""
    B, dk, dv = (1 << 17) + 8, 128, 128
    off = np.array([0, 3], dtype=np.int32)
    lay = DecodeLayer("gdn", B, 1, 1, dk, dv, 1, act, act, off)
    assert lay.S.numel() > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(95)
    lay.Pt.copy_(torch.randn(lay.Pt.shape, generator=g, device="cuda") / dk ** 0.5)
    lay.Cmap.copy_(lay.Pt)
    ends = [0, B - 1]
    for b in ends:
        lay.S[b] = 0.1 * torch.randn(lay.S[b].shape, generator=g, device="cuda")
    tok = make_tokens(2 * n, 1, dk, dv, act, seed=96, alpha=1 - 0.001 * torch.rand((2 * n, 1), generator=g, device="cuda"))
    first = {b: f64(lay.S[b]) for b in ends}
    _, starts = run(lay, tok, [n, n], seqs=ends)
    assert lay.error_word() == 0
    t64 = [f64(x) for x in tok]
    for i, b in enumerate(ends):
        sl = slice(i * n, (i + 1) * n)
        o, S, top = ref.delta_rule(t64[0][sl, 0], t64[1][sl, 0], t64[2][sl, 0], t64[3][sl, 0], t64[4][sl, 0], first[b][0])
        # as in check: (dk + 8) roundings of 2^-24 a token of the largest column norm
        lim = n * (dk + 8) * EPS32 * top
        assert np.abs(f64(lay.S[b, 0]) - S).max() <= lim
    assert not lay.S[1:B - 1:4096].any()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_a_long_prompt_among_empty_ones(dk, dv, act):
    """As many tokens as prompts, as a decode batch has, but most in one prompt."""
    n, lens = 150, [0] * 150
    lens[3], lens[70], lens[149] = 1, 130, 2
    lay = make_layer(n, 2, dk, dv, act, seed=97)
    tok = make_tokens(n, 2, dk, dv, act, seed=98)      # (rows behind the last prompt's end)
    S0 = lay.S.clone()
    has = [i % 2 for i in range(n)]
    _, starts = run(lay, tok, lens, has=has)
    assert lay.error_word() == 0
    check(lay, S0, tok, lens, starts, list(range(n)), has)
