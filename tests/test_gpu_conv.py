"""The short causal convolution against its definition in 64 bits.  Tolerances: a
sum of taps products and a bias takes taps + 1 roundings of 2^-24 of its terms'
magnitudes, an activation (no steeper than 1.1) some units of its result (bf16: the
exponential of a rounded argument, 2^-24 |y|), a head's length its sum's dk
roundings and its elements' own; then one rounding to the type."""
import numpy as np
import pytest
import torch

from tests import sequence_ref as ref

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.layer import DecodeLayer, TORCH_DTYPE
    from ssm_decode_amd.serving import ShortConv


def f64(x):
    return x.double().cpu().numpy()


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, N, B, family="mamba2", H=6, G=2, dk=64, dv=64, act="bf16", taps=4, fn="silu", order="vkq", unit=False,
                 bias=True, pad=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        d = TORCH_DTYPE[act]
        self.lay = DecodeLayer(family, B, H, G, dk, dv, 4, act, act, np.arange(H + 1) * 2)
        self.act, self.fn, self.order, self.dk = act, fn, order, dk
        self.sizes = {"q": G * dk, "k": G * dk, "v": H * dv}
        C = sum(self.sizes.values())
        w = rand(C, taps) / taps ** 0.5
        self.conv = ShortConv(self.lay, w, 0.3 * rand(C) if bias else None, act=fn, order=order, unit=unit)
        self.conv.state.copy_(rand(*self.conv.state.shape))
        self.held = self.conv.state.clone()
        self.x = rand(N, C + 2 * pad).to(d)[:, pad:pad + C]
        self.y = torch.full((N, C + pad), 5.0, device="cuda", dtype=d)
        at, self.out = 0, {}
        for c in order:
            shape = (G, dk) if c != "v" else (H, dv)
            self.out[c] = self.y[:, at:at + self.sizes[c]].unflatten(1, shape)
            at += self.sizes[c]

    def call(self, **kw):
        return self.lay.convolve(self.conv, self.x, self.out["q"], self.out["k"], self.out["v"], **kw)

    def check(self, at, seqs, has):
        x, held, w = f64(self.x), f64(self.held), f64(self.conv.weight)
        b = f64(self.conv.bias) if self.conv.bias is not None else np.zeros(len(w))
        taps, half = w.shape[1], ref.HALF[self.act]
        got = {c: f64(t) for c, t in self.out.items()}
        state = f64(self.conv.state)
        done = np.zeros(len(x), bool)
        for i, s in enumerate(seqs):
            rows = slice(at[i], at[i + 1])
            done[rows] = True
            y, out, m, after = ref.conv(x[rows], held[s] * has[i], w, b, self.fn)
            units = 8 if self.act == "f32" else 16 + 2 * np.abs(y)
            tol = ref.U * (1.1 * (taps + 1) * m + (units * np.abs(out) if self.fn != "none" else 0))
            first = 0
            for c in self.order:
                n = self.sizes[c]
                z, t = out[:, first:first + n], tol[:, first:first + n]
                if self.conv.unit and c != "v":
                    z, t = (u.reshape(len(u), n // self.dk, self.dk) for u in (z, t))
                    norm = np.sqrt((z ** 2).sum(-1, keepdims=True) + 1e-6)
                    t = t / norm + np.abs(z) / norm * ((np.abs(z) * t).sum(-1, keepdims=True) / norm ** 2 + (self.dk + 8) * ref.U)
                    z = z / norm
                d = np.abs(got[c][rows].reshape(z.shape) - z)
                assert (d <= half * np.abs(z) + 1.01 * t).all(), (c, i, d.max())
                first += n
            assert (state[s] == after).all()
        for s in set(range(self.lay.B)) - set(seqs):
            assert (state[s] == held[s]).all()
        assert (f64(self.y)[~done] == 5).all() and (f64(self.y)[:, sum(self.sizes.values()):] == 5).all()
        assert self.conv.error_word() == 0


LENS = [1, 0, 2, 3, 70, 0, 33, 129, 32, 5]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("taps", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("shape", [dict(), dict(unit=True), dict(H=5, G=1, dk=128, dv=64, unit=True, order="qkv"),
                                   dict(family="gdn", H=3, G=3, dk=128, dv=128, unit=True, order="kqv"),
                                   dict(H=2, G=1, dk=16, dv=32, unit=True, fn="none", bias=False),
                                   dict(H=22, G=2, dk=128, dv=64, fn="sigmoid")])
def test_prompts(shape, taps, act):
    n = len(LENS)
    c = Case(sum(LENS) + 4, n + 2, act=act, taps=taps, seed=taps, **shape)
    at = [1 + sum(LENS[:i]) for i in range(n + 1)]
    seqs, has = [(5 * i + 2) % (n + 2) if (n + 2) % 5 else n - i for i in range(n)], [i % 3 != 1 for i in range(n)]
    assert c.call(seq_start=ints(at), seqs=ints(seqs), has_state=ints(has)) == 0
    c.check(at, seqs, has)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("B", [1, 7, 64, 702])
@pytest.mark.parametrize("taps", [2, 4])
def test_single_tokens(B, taps, act):
    c = Case(B, B, act=act, taps=taps, unit=True, H=4, G=2, dk=128, dv=64, seed=B)
    assert c.call() == 0
    c.check(range(B + 1), range(B), [1] * B)
    # some of the sequences, in another order, some of them anew
    n = max(1, B // 2)
    c = Case(n, B, act=act, taps=taps, seed=B + 1)
    seqs, has = [B - 1 - 2 * i for i in range(n)], [i % 2 for i in range(n)]
    assert c.call(seqs=ints(seqs), has_state=ints(has)) == 0
    c.check(range(n + 1), seqs, has)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("n", [641, 703])
def test_many_single_tokens(n, act):
    """Workgroups of four tokens each; sequences in another order, refused ones among them."""
    B = n + 5
    c = Case(n, B, act=act, unit=True, H=2, G=1, dk=64, dv=64, seed=n)
    seqs, has = [B - 1 - i for i in range(n)], [int(i % 3 > 0) for i in range(n)]
    assert c.call(seqs=ints(seqs), has_state=ints(has)) == 0
    c.check(range(n + 1), seqs, has)
    c = Case(n, B, act=act, unit=True, H=2, G=1, dk=64, dv=64, seed=n + 1)
    seqs[3], seqs[n - 1], seqs[9] = B, seqs[0], -1       # outside, listed before, outside
    assert c.call(seqs=ints(seqs), has_state=ints(has)) == 0
    assert c.conv.error_word() == 4
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[3, 9, n - 1]] = True
    assert ((c.y[:, :256] == 5).all(1) == bad).all()
    kept = sorted(set(range(B)) - {x for i, x in enumerate(seqs) if i not in (3, 9, n - 1)})
    same = (c.conv.state == c.held).flatten(1).all(1)
    assert torch.nonzero(same).flatten().tolist() == kept


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_prompt_is_its_tokens(act):
    """Token by token, in two calls and in one: the same bits."""
    T, outs = 75, []
    for cuts in ([75], [40, 75], list(range(1, 76))):
        c = Case(T, 1, act=act, unit=True, seed=3)
        a = 0
        for b in cuts:
            kw = dict(seq_start=ints([0, b - a])) if b - a > 1 else {}
            assert c.lay.convolve(c.conv, c.x[a:b], *(c.out[n][a:b] for n in "qkv"), **kw) == 0
            a = b
        outs.append((c.y.clone(), c.conv.state.clone()))
    for y, s in outs[1:]:
        assert torch.equal(y, outs[0][0]) and torch.equal(s, outs[0][1])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_stay_in_their_reach(value):
    c, d = Case(100, 1, unit=True, seed=4), Case(100, 1, unit=True, seed=4)
    first = c.sizes["v"] + 64 + 3                      # of the second head of keys
    c.x[40, first] = value
    c.x[60, 5] = value
    c.held[0, 1, 9] = value
    c.conv.state.copy_(c.held)
    for z in (c, d):
        assert z.call(seq_start=ints([0, 100])) == 0
    wrong = torch.zeros_like(c.y, dtype=torch.bool)
    wrong[40:44, c.sizes["v"] + 64:c.sizes["v"] + 128] = True
    wrong[60:64, 5] = True
    wrong[:2, 9] = True
    assert torch.equal(c.y[~wrong], d.y[~wrong])
    assert not torch.isfinite(c.y[40:44, first].float()).any() or value < 0


@pytest.mark.parametrize("step", [False, True])
def test_refusals_on_the_device(step):
    def call(seqs, start=None, n=3):
        c = Case(n, 4, seed=5)
        kw = dict(seqs=ints(seqs)) if step else dict(seqs=ints(seqs), seq_start=ints(start))
        assert c.call(**kw) == 0
        same = [bool(torch.equal(c.conv.state[b], c.held[b])) for b in range(4)]
        return c.conv.error_word(), same, [bool((c.y[t] == 5).all()) for t in range(n)]

    s = [0, 1, 2, 3]
    assert call([0, 1, 3], s) == (0, [False, False, True, False], [False] * 3)
    assert call([0, 4, 3], s) == (4, [False, True, True, False], [False, True, False])
    assert call([0, -1, 3], s) == (4, [False, True, True, False], [False, True, False])
    assert call([2, 1, 2], s) == (4, [True, False, False, True], [False, False, True])
    if not step:
        for bad in ([0, 2, 1, 3], [0, 1, 2, 4], [-1, 1, 2, 3], [900] * 4):
            assert call([0, 1, 2], bad) == (4, [True] * 4, [True] * 3)


def test_captured_and_replayed():
    c = Case(300, 3, seed=6)
    st = ints([0, 100, 100, 300])
    c.call(seq_start=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert c.call(seq_start=st) == 0
    for at in ([0, 7, 200, 299], [0, 100, 100, 300], [3, 3, 3, 250]):
        st.copy_(ints(at))
        c.y.fill_(5)
        c.conv.state.copy_(c.held)
        g.replay()
        torch.cuda.synchronize()
        c.check(at, [0, 1, 2], [1, 1, 1])
