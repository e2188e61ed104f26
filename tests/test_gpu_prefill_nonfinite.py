"""An infinity or a NaN in a prompt: outputs and states are no finite numbers
where the recurrence's are none, and right everywhere else; no earlier token
sees it."""
import pytest
import torch

from tests.prompt_bounds import EPS32, rule, wrong_outputs
from tests.test_gpu_prefill import make_layer, make_tokens, run

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def put(tok, S, what, t, h, value):
    """One value of token t, head h (of the state: of a column)."""
    if what == "state":
        S[h, 3, 21] = value
    elif what in ("gate", "beta"):
        tok[3 if what == "gate" else 4][t, h] = value
    else:
        tok["qkv".index(what)][t, h, 9] = value


def compare(lay, b, S0, tok, part, has=True):
    """Prompt `part` of the tokens, sequence b, against the recurrence."""
    o, S, scale = rule(*(x[part] for x in tok[:5]), S0 if has else torch.zeros_like(S0))
    got, fine = tok[5][part], torch.isfinite(o)
    assert torch.equal(torch.isfinite(got.float()), fine)
    zero = torch.zeros_like(o)
    assert wrong_outputs(torch.where(fine, got, zero.to(got.dtype)), torch.where(fine, o, zero),
                         torch.where(fine, scale, zero), lay.dk) == (0, 0)
    assert torch.equal(torch.isfinite(lay.S[b]), torch.isfinite(S))
    for h in range(lay.H):                        # the columns that stay finite
        c = torch.isfinite(S[h]).all(0)
        d = (lay.S[b, h][:, c].double() - S[h][:, c]).norm()
        assert d <= 8 * lay.dk ** 0.5 * EPS32 * S[h][:, c].norm()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 32), (64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("what", ["q", "k", "v", "gate", "beta", "state"])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_nothing_reaches_an_earlier_token(act, dk, dv, what, value):
    """At the ends and in the middle of chunks, in the last chunk's, in the last
    token, which the rows behind the end repeat."""
    H, lens, at = 2, [150, 150, 150, 150, 150, 90], [0, 37, 63, 64, 149, 80]
    n = len(lens)
    lay = make_layer(n, H, dk, dv, act, seed=500, ranks=[3, 0])
    tok = make_tokens(sum(lens), H, dk, dv, act, seed=501, packed=True)
    starts = [sum(lens[:i]) for i in range(n)]
    for i in range(n):
        put(tok, lay.S[i], what, starts[i] + at[i], i % H, value)
    S0 = lay.S.clone()
    run(lay, tok, lens)
    assert lay.error_word() == 0
    for i in range(n):
        compare(lay, i, S0[i], tok, slice(starts[i], starts[i] + lens[i]))


@pytest.mark.parametrize("what", ["q", "k", "v", "gate", "beta", "state"])
@pytest.mark.parametrize("at", [5, 511, 512, 1900, 2147])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_in_segments(dk, dv, what, at):
    lay = make_layer(2, 3, dk, dv, "bf16", seed=502)
    tok = make_tokens(2148, 3, dk, dv, "bf16", seed=503)
    put(tok, lay.S[0], what, at, 1, NAN)
    S0 = lay.S.clone()
    run(lay, tok, [2148], seqs=[0])
    compare(lay, 0, S0[0], tok, slice(0, 2148))
    assert torch.equal(lay.S[1], S0[1])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_several_in_one_prompt(act):
    """Columns that turn at different tokens, and a key behind them."""
    lay = make_layer(1, 2, 128, 128, act, seed=504)
    tok = make_tokens(400, 2, 128, 128, act, seed=505)
    for t, c in ((300, 0), (20, 1), (130, 1), (131, 17), (64, 127), (399, 64)):
        tok[2][t, 0, c] = INF
    tok[2][200, 1, 40] = NAN
    tok[1][260, 1, 0] = NAN
    tok[0][10, 1, 0] = NAN
    S0 = lay.S.clone()
    run(lay, tok, [400])
    compare(lay, 0, S0[0], tok, slice(0, 400))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_an_overflow_reaches_back_to_its_own_chunk_at_most(act):
    """A column of 2^127 whose product with a late key overflows, beside one that
    has had a NaN since the first chunk, or has one later."""
    for early, late in ((10, None), (None, 250), (10, 250)):
        lay = make_layer(1, 1, 64, 64, act, seed=506, ranks=[0])
        q, k, v, al, be, o = make_tokens(300, 1, 64, 64, act, seed=507)
        lay.S[:, :, :, 7] = 2.0 ** 127
        k.zero_()
        k[:, 0, 0], k[:, 0, 1] = 0.75, -0.75       # nothing of it, but for token 200
        k[200, 0, :4] = 0.75
        q.mul_(2.0 ** -10)
        al.fill_(1.0)
        be.zero_()
        if early is not None:
            v[early, 0, 3] = NAN
        if late is not None:
            v[late, 0, 7] = NAN
        want = torch.einsum("tk,kc->tc", q[:, 0].double(), lay.S[0, 0].double())
        run(lay, (q, k, v, al, be, o), [300])
        got = o[:, 0].double()
        assert torch.isfinite(got[:192, 7]).all() and not torch.isfinite(got[200:, 7]).any()
        assert ((got[:192, 7] - want[:192, 7]).abs() <= 2.0 ** -7 * want[:192, 7].abs() + 2.0 ** 127 * 64 * 2.0 ** -34 * 8).all()
        fine = torch.isfinite(got[:, 3])
        assert fine.tolist() == [early is None or t < early for t in range(300)]
        others = [c for c in range(64) if c not in (3, 7)]
        assert torch.isfinite(got[:, others]).all() and torch.isfinite(lay.S[0, 0][:, others]).all()
        assert not torch.isfinite(lay.S[0, 0, :, 7]).any()
