"""The outputs of prompts in chunks are products of fp32 operands: outputs
that are the small difference of two large terms show every bit that an
operand is short of."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests.test_gpu_prefill import EPS32, SHAPES, f64, make_layer, make_tokens, run

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -12      # the pair's relative difference


def compare(lay, tok, S0, terms):
    """|o - exact| <= half a step of the type + 2^-24 of the two terms for each
    rounding: `terms` [N, H, dv] counts roundings times |terms|."""
    q, k, v, al, be, _ = [f64(x) for x in tok]
    half = torch.finfo(tok[5].dtype).eps / 2
    got = f64(tok[5])
    for h in range(lay.H):
        o, _, _ = ref.delta_rule(q[:, h], k[:, h], v[:, h], al[:, h], be[:, h], S0[h])
        assert np.abs(o).max() > 0
        assert (np.abs(got[:, h] - o) <= half * np.abs(o) * (1 + half) + EPS32 * terms[:, h]).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES[1:])
def test_the_state_read_by_queries_has_all_its_bits(dk, dv, act):
    """o = q (S_a + S_b) with S_b about -S_a, the state unchanged (beta 0, no
    decay).  Of each row of S reaches the sum: two products, each of at most
    three exact parts, in at most eight sums; with the factor one and the second
    chunk's state (unchanged) 16 roundings are more than there are."""
    N, H = 130, 2
    lay = make_layer(1, H, dk, dv, act, seed=200)
    lay.S[:, :, 1::2] = -lay.S[:, :, 0::2] * (1 + STEP)
    q, k, v, al, be, o = make_tokens(N, H, dk, dv, act, seed=201)
    al.fill_(1.0)
    be.zero_()
    at = 2 * (torch.arange(N, device="cuda") % (dk // 2))
    x = q[:, :, :1].clone()
    q.zero_()
    q.scatter_(2, at[:, None, None].expand(N, H, 1), x)
    q.scatter_(2, (at + 1)[:, None, None].expand(N, H, 1), x)
    S0 = f64(lay.S)[0]
    tok = (q, k, v, al, be, o)
    run(lay, tok, [N])
    terms = 16 * np.einsum("thi,hic->thc", np.abs(f64(q)), np.abs(S0))
    compare(lay, tok, S0, terms)


@pytest.mark.parametrize("operand", ["values", "products"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES[1:])
def test_the_tokens_of_a_chunk_read_by_queries_have_all_their_bits(dk, dv, act, operand):
    """o_i = q_i (D_ia u_a + D_ib u_b) within a chunk, keys of one element each.
    "values": u_b about -u_a by their betas, no decay; "products": u_b = -u_a, the
    decay between a and b makes the difference and further ones fill the bits
    of D.  Roundings: each decay's product, and 16 as above."""
    N, H = 64, 2
    lay = make_layer(1, H, dk, dv, act, seed=202)
    q, k, v, al, be, o = make_tokens(N, H, dk, dv, act, seed=203)
    k.zero_()
    k[torch.arange(N), :, torch.arange(N)] = 1
    v[1::2] = -v[0::2]
    if operand == "values":
        al.fill_(1.0)
        be[1::2] = be[0::2] * (1 + STEP)
    else:
        al[1::2] = 1 - STEP
        be.fill_(1.0)
    i = torch.arange(N, device="cuda")
    a = 2 * torch.clamp((i - 1) // 2 - i % 7, min=0)          # (token 0 reads its own value alone)
    x = q[:, :, :1].clone()
    q.zero_()
    q.scatter_(2, a[:, None, None].expand(N, H, 1), x)
    q.scatter_(2, (a + 1)[:, None, None].expand(N, H, 1), x)
    tok = (q, k, v, al, be, o)
    run(lay, tok, [N], has=[0])
    S0 = np.zeros((H, dk, dv))
    qq, vv, bb, n = f64(q), np.abs(f64(v)), f64(be), (i - a).cpu().numpy()
    both = sum(np.abs(qq[np.arange(N), :, c])[:, :, None] * bb[c][:, :, None] * vv[c]
               for c in (a.cpu().numpy(), a.cpu().numpy() + 1))
    compare(lay, tok, S0, (n + 16)[:, None, None] * both)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES[1:])
def test_the_triangular_product_keeps_what_reaches_2_to_minus_24(dk, dv, act):
    """Keys of one element each, no values, no decay: row j of the state becomes
    S - beta S, of which the operands' low bits are a good part.  Roundings of
    2^-24 of S: the product's, its two lower parts' sums with S (the last sum is
    exact), one for the product's terms that may be left out: four, by a factor
    that is under 1 + 2^-6."""
    N, H = 64, 2
    lay = make_layer(1, H, dk, dv, act, seed=204)
    ones = 1 + 2.0 ** -7 - 2.0 ** -23           # eight bits 1.0000000, then ones throughout
    lay.S.copy_(torch.sign(lay.S) * ones * torch.exp2(torch.floor(50 * lay.S)))
    q, k, v, al, be, o = make_tokens(N, H, dk, dv, act, seed=205)
    k.zero_()
    k[torch.arange(N), :, torch.arange(N)] = 1
    v.zero_()
    al.fill_(1.0)
    be.fill_(ones)
    S0 = f64(lay.S)
    run(lay, (q, k, v, al, be, o), [N])
    want = S0.copy()
    want[:, :, :N] -= float(be[0, 0]) * S0[:, :, :N]
    assert (np.abs(f64(lay.S) - want) <= 4 * EPS32 * (1 + 2.0 ** -6) * np.abs(S0)).all()
