"""The selection of beams against its definition in 64 bits, and the reordering of
sequences bit for bit.  Parents and tokens are compared exactly: the inputs' best
candidates are further apart than the sums' errors (checked).  A score is rounded
to fp32 once, behind a logarithm of a sum of V exponentials in fp32, whose
relative error (2^-22 each with its argument, and the sum's log2 V + 64 roundings
along its tree) is the logarithm's absolute one."""
import numpy as np
import pytest
import torch

from tests import sequence_ref as ref

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.layer import DecodeLayer, TORCH_DTYPE
    from ssm_decode_amd.serving import BeamSearch, ShortConv

INF = float("inf")
LOGIT, SEQ = 16, 4
TOL = 2.0 ** -16                     # (64 + 17 roundings of 2^-24, and 2^-20)


def f64(x):
    return x.double().cpu().numpy()


def inputs(n, k, V, act, seed=0, scale=2.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (scale * torch.randn((n * k, V + pad), generator=g, device="cuda")).to(TORCH_DTYPE[act])[:, :V]
    s = -5 * torch.rand((n, k), generator=g, device="cuda")
    return x, s


def check(search, x, scores, ended, err=0):
    n, k = scores.shape
    want = ref.beams(f64(x).reshape(n, k, -1), f64(scores), ended.cpu().numpy(), search.end)
    assert (search.parents.cpu().numpy() == want[0]).all()
    assert (search.tokens.cpu().numpy() == want[1]).all()
    got, fine = f64(search.scores), np.isfinite(want[2])
    assert (np.isneginf(got) == ~fine).all()
    assert (np.abs(got - want[2])[fine] <= (2.0 ** -24 * np.abs(want[2]) + TOL)[fine]).all()
    assert (search.ended.cpu().numpy() == want[3]).all()
    assert search.error_word() == err


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,V,pad", [(1, 1, 1, 0), (2, 4, 3, 0), (3, 16, 5, 3), (3, 5, 97, 1), (1, 4, 4099, 0), (2, 16, 8192, 8), (5, 3, 50001, 0),
                                       (1, 8, 128000, 0), (40, 2, 1000, 7), (2, 16, 100000, 0), (1, 16, 170001, 3)])
def test_selection(n, k, V, pad, act):
    x, s = inputs(n, k, V, act, seed=V, pad=pad)
    search = BeamSearch(n, k, V, end=V - 1)
    none = torch.zeros_like(search.ended)
    assert search.select(x, s, none) == 0
    check(search, x, s, none)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_first_step_has_one_beam(act):
    x, _ = inputs(4, 5, 700, act, seed=1)
    search = BeamSearch(4, 5, 700)
    s, e = search.scores.clone(), search.ended.clone()
    assert search.select(x) == 0
    check(search, x, s, e)
    assert (search.parents == 5 * torch.arange(4, device="cuda")[:, None]).all()
    s, e = search.scores.clone(), search.ended.clone()
    x, _ = inputs(4, 5, 700, act, seed=2)
    assert search.select(x) == 0                  # in place
    check(search, x, s, e)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("k,V", [(4, 900), (14, 900), (14, 60000)])
def test_ended_beams_and_ruled_out_tokens(k, V, act):
    n = 6
    x, s = inputs(n, k, V, act, seed=3)
    ended = torch.zeros((n, k), dtype=torch.int32, device="cuda")
    ended[0, 1] = ended[1, 0] = 7
    ended[2] = 1                                  # all of them
    x[3 * k:4 * k] = -INF                         # nothing is left
    x[4 * k + 1:5 * k] = -INF                     # one beam is left ..
    x[4 * k, 2:] = -INF                           # .. with two tokens
    s[5, 0] = -INF
    x[:, ::3] = -INF
    x[0, 17] = torch.finfo(x.dtype).min
    search = BeamSearch(n, k, V, end=17)
    assert search.select(x, s, ended) == 0
    check(search, x, s, ended)
    assert (search.tokens[3] == -1).all() and (search.tokens[2] == 17).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("value", [0.0, -0.0, 3.0, -1e30])
@pytest.mark.parametrize("n,k,V", [(2, 6, 40000), (2, 16, 40000), (1, 16, 170000)])
def test_ties_go_to_the_lowest_index(n, k, V, value, act):
    """All logits alike: every wave's and part's list is full of ties."""
    x = torch.full((n * k, V), value, device="cuda", dtype=TORCH_DTYPE[act])
    x[:, 1::2] *= -1 if value == 0 else 1
    s = torch.zeros((n, k), device="cuda")
    search = BeamSearch(n, k, V)
    assert search.select(x, s, torch.zeros_like(search.ended)) == 0
    assert (search.parents == k * torch.arange(n, device="cuda")[:, None]).all()
    assert (search.tokens == torch.arange(k, device="cuda")).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), INF])
@pytest.mark.parametrize("k", [4, 9])
def test_wrong_logits_take_their_beam_out(k, value, act):
    x, s = inputs(3, k, 5000, act, seed=5)
    clean = x.clone()
    x[k + 1, 4321] = value
    x[k + 1, 7] = value
    search = BeamSearch(3, k, 5000)
    e = torch.zeros_like(search.ended)
    assert search.select(x, s, e) == 0
    out = s.clone()
    out[1, 1] = -INF
    check(search, clean, out, e, err=LOGIT)
    search = BeamSearch(3, k, 5000)
    wrong = s.clone()
    wrong[1, 1] = value
    assert search.select(clean, wrong, e) == 0
    check(search, clean, out, e, err=LOGIT)


def test_captured_and_replayed():
    n, k, V = 3, 4, 30011
    x, s = inputs(n, k, V, "bf16", seed=6)
    search = BeamSearch(n, k, V, end=5)
    e = torch.zeros_like(search.ended)
    search.select(x, s, e)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert search.select(x, s, e) == 0
    for seed in (7, 8, 9):
        x.copy_(inputs(n, k, V, "bf16", seed=seed)[0])
        g.replay()
        torch.cuda.synchronize()
        check(search, x, s, e)


def test_rows_far_apart():
    x, s = inputs(1, 4, 1000, "f32", seed=10)
    far = torch.empty(3 * (1 << 30) + 1000, device="cuda").as_strided((4, 1000), (1 << 30, 1))
    far.copy_(x)
    search = BeamSearch(1, 4, 1000)
    e = torch.zeros_like(search.ended)
    assert search.select(far, s, e) == 0
    check(search, x, s, e)


# ------------------------------------------------------------- reordering
LAYERS = [("mamba2", dict(H=3, G=3, dk=16, dv=32, W=5, act="bf16")), ("mamba2", dict(H=6, G=2, dk=128, dv=64, W=16, act="bf16")),
          ("gdn", dict(H=3, G=3, dk=64, dv=64, W=3, act="f32", pullback="proj")),
          ("kda", dict(H=2, G=2, dk=128, dv=128, W=4, act="bf16", coef="state"))]


def make(family, B, H, G, dk, dv, W, act, seed=0, dense=True, **kw):
    ranks = [0 if dense and h == 1 else 3 for h in range(H)]
    lay = DecodeLayer(family, B, H, G, dk, dv, W, act, act, np.concatenate([[0], np.cumsum(ranks)]), **kw)
    conv = ShortConv(lay, torch.zeros(2 * G * dk + H * dv, 4, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(seed)
    held = {}
    for name in ("S", "U", "Cstate", "Scopy", "ring_k", "ring_v", "ring_gate", "ring_beta", "ring_pc", "count"):
        x = getattr(lay, name)
        if x is not None:
            x.copy_(torch.randint(0, 9, x.shape, generator=g, device="cuda"))
            held[name] = x
    conv.state.copy_(torch.randn(conv.state.shape, generator=g, device="cuda"))
    held["conv"] = conv.state
    return lay, conv, held


@pytest.mark.parametrize("family,kw", LAYERS)
@pytest.mark.parametrize("groups,k", [(1, 1), (3, 2), (2, 4), (2, 7), (1, 16)])
def test_reorder(family, kw, groups, k):
    B = groups * k
    g = torch.Generator(device="cuda").manual_seed(k)
    for parents in (torch.randint(0, k, (groups, k), generator=g, device="cuda"), torch.arange(k, device="cuda").flip(0).expand(groups, k),
                    torch.full((groups, k), k - 1, device="cuda"), torch.arange(k, device="cuda").expand(groups, k),
                    torch.arange(k, device="cuda").roll(1).expand(groups, k)):
        lay, conv, held = make(family, B, seed=k, **kw)
        at = (parents + k * torch.arange(groups, device="cuda")[:, None]).to(torch.int32)
        want = {n: x[at.flatten().long()].clone() for n, x in held.items()}
        still = (lay.Pt.clone(), lay.Cmap.clone(), lay.offsets.clone())
        assert lay.reorder(at, k, convs=(conv,)) == 0
        for n, x in held.items():
            assert torch.equal(x, want[n]), n
        assert all(torch.equal(a, b) for a, b in zip(still, (lay.Pt, lay.Cmap, lay.offsets)))
        assert lay.error_word() == 0


def test_a_parent_outside_its_group():
    for bad in (3, -1, 6, 2 ** 30):
        lay, conv, held = make("mamba2", 6, H=2, G=1, dk=64, dv=64, W=4, act="bf16", seed=1)
        before = {n: x.clone() for n, x in held.items()}
        at = torch.tensor([1, 0, bad, 4, 4, 4], dtype=torch.int32, device="cuda")
        assert lay.reorder(at, 3, convs=(conv,)) == 0
        for n, x in held.items():
            assert torch.equal(x[:3], before[n][:3]) and torch.equal(x[3:], before[n][[4, 4, 4]]), n
        assert lay.error_word() == SEQ


def test_reorder_captured_and_replayed():
    lay, conv, held = make("mamba2", 8, H=4, G=2, dk=64, dv=64, W=4, act="bf16", seed=2)
    at = torch.arange(8, dtype=torch.int32, device="cuda")
    lay.reorder(at, 4, convs=(conv,))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert lay.reorder(at, 4, convs=(conv,)) == 0
    for new in ([1, 0, 3, 2, 4, 4, 4, 4], [3, 3, 0, 0, 7, 6, 5, 4], [0, 0, 0, 0, 5, 6, 7, 4]):
        want = {n: x[new].clone() for n, x in held.items()}
        at.copy_(torch.tensor(new))
        g.replay()
        torch.cuda.synchronize()
        for n, x in held.items():
            assert torch.equal(x, want[n]), n
