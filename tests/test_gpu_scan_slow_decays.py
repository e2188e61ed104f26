"""Prompts of slow, steady decays, token by token, against the sums in 64 bits.

A token's two roundings of the state, at most 2^-24 of an element each and of either
sign, fade as the state does: those of n = min(T, 1 / (2 l)) tokens count (l the decay's
logarithm), in quadrature 2^-24 sqrt(2 n) of the state.  Allowed is twice that, and 16
units more for the decays' own errors (a few units of l each, which over the 1 / l tokens
that count come to as many of the state), the segments' joins and an output's sum.  It does not
grow with the prompt, as the worst case of the roundings would."""
import numpy as np
import pytest
import torch

from tests.test_gpu_scan import ints, make_layer, make_tokens, starts

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.serving import ScanPrompts


def steady(q, k, v, l, dt, S):
    """One head's outputs and last state in 64 bits: q, k [T, dk], v [T, dv], decays exp(-l) a token."""
    o, C = torch.empty_like(v), 1000
    for t in range(0, len(v), C):
        Q, K, V = q[t:t + C], k[t:t + C], v[t:t + C] * dt
        i = torch.arange(len(V), device=v.device, dtype=torch.float64)
        D = torch.exp(-l * (i[:, None] - i[None, :]).clamp(min=0)).tril()
        o[t:t + C] = torch.exp(-l * (i + 1))[:, None] * (Q @ S) + (Q @ K.T.contiguous() * D) @ V
        S = np.exp(-l * len(V)) * S + (K * torch.exp(-l * (len(V) - 1 - i))[:, None]).T.contiguous() @ V
    return o, S


def off(x, y):
    return float((x.double() - y).norm() / y.norm())


@pytest.mark.parametrize("T,dt", [(4000, 1e-3), (16000, 3e-4), (16000, 2e-5)])
@pytest.mark.parametrize("n,H,G,dk,dv,act", [(1, 2, 1, 64, 64, "f32"), (2, 3, 3, 16, 32, "f32"), (1, 2, 1, 128, 128, "f32"),
                                             (33, 16, 1, 128, 64, "f32"), (1, 2, 2, 16, 32, "bf16"), (1, 2, 1, 64, 64, "bf16"),
                                             (33, 16, 1, 128, 64, "bf16"), (2, 4, 4, 128, 128, "bf16")])
def test_slow_steady_decays(n, H, G, dk, dv, act, T, dt):
    """n > 1: the others are short; 33 of 16 heads are too many states for segments."""
    lens = [T] + [3] * (n - 1)
    N = sum(lens)
    lay = make_layer(n, H, G, dk, dv, act, seed=600)
    q, k, v, d, o = make_tokens(N, H, G, dk, dv, act, seed=601)
    d.fill_(dt)
    lay.S[0].zero_()
    lay.A.copy_(torch.log(torch.tensor([1.0, 2.5], device="cuda")).repeat(H)[:H])
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    assert lay.scan(ScanPrompts(lay, q, k, v, d, o, ints(at))) == 0
    step = float(d[0, 0].double())
    for h in {0, H - 1}:
        g, l = h // (H // G), step * float(torch.exp(lay.A[h].double()))
        oo, SS = steady(q[:T, g].double(), k[:T, g].double(), v[:T, h].double(), l, step, torch.zeros_like(lay.S[0, h], dtype=torch.float64))
        bound = 2.0 ** -24 * (2 * (2 * min(T, 1 / (2 * l))) ** 0.5 + 16)
        assert off(lay.S[0, h], SS) <= bound, (h, off(lay.S[0, h], SS) / bound)
        if act == "f32":
            assert off(o[:T, h], oo) <= bound, (h, off(o[:T, h], oo) / bound)
    assert lay.error_word() == 0


@pytest.mark.parametrize("A", [95.0, 800.0])
@pytest.mark.parametrize("lens", [[3, 1, 20], [70, 5, 130]])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_rates_past_the_types_end(act, lens, A):
    """exp(A) past fp32's end, and past that of 64 bits: every step forgets all, and one of 0 nothing."""
    n, N = len(lens), sum(lens)
    lay = make_layer(n, 4, 2, 64, 64, act, seed=610)
    q, k, v, d, o = make_tokens(N, 4, 2, 64, 64, act, seed=611)
    lay.A[1::2] = A
    d[::3] = 0
    S0 = lay.S.double()
    assert lay.scan(ScanPrompts(lay, q, k, v, d, o, ints(starts(lens)))) == 0
    at, unit = starts(lens), 2.0 ** -24
    for i in range(n):
        s = slice(at[i], at[i + 1])
        for h in (1, 3):
            S, K, Q = S0[i, h].clone(), k[s, h // 2].double(), q[s, h // 2].double()
            V, D = v[s, h].double(), d[s, h].double()
            for t in range(lens[i]):
                S = (S if D[t] == 0 else 0 * S) + D[t] * K[t][:, None] * V[t][None, :]
                want = (Q[t][:, None] * S).sum(0)
                off = 300 * unit * (Q[t].abs()[:, None] * S.abs()).sum(0) + (2.0 ** -8 if act == "bf16" else unit) * want.abs()
                assert bool(((o[at[i] + t, h].double() - want).abs() <= off).all()), (i, h, t)
            assert bool(((lay.S[i, h].double() - S).abs() <= 16 * unit * S.abs()).all()), (i, h)
    assert lay.error_word() == 0
