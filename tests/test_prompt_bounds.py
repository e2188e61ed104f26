"""The bounds of long prompts' outputs, on the CPU: they take what rounding
gives and nothing else."""
import pytest
import torch

from tests.prompt_bounds import rule, state_off, wrong_outputs

T, H, SEG = 2100, 2, 512


def tokens(dk, dv, decay):
    g = torch.Generator().manual_seed(7)
    unit = lambda *s: torch.nn.functional.normalize(torch.randn(s, generator=g), dim=-1).bfloat16()  # noqa: E731
    q, k = unit(T, H, dk), unit(T, H, dk)
    v = (torch.randn((T, H, dv), generator=g) / dv ** 0.5).bfloat16()
    al = 1 - decay * torch.rand((T, H), generator=g)
    be = torch.rand((T, H), generator=g)
    return q, k, v, al, be, 0.1 * torch.randn((H, dk, dv), generator=g)


def in_segments(tok, S, start):
    """The prompt as segments that start from start(segment, state before it)."""
    out = []
    for j, a in enumerate(range(0, T, SEG)):
        o, S, _ = rule(*(x[a:a + SEG] for x in tok), start(j, S))
        out.append(o)
    return torch.cat(out)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("decay", [0.001, 0.1])
def test_planted_mistakes_are_found(dk, dv, decay):
    *tok, S0 = tokens(dk, dv, decay)
    o, S, scale = rule(*tok, S0)
    for dtype in (torch.bfloat16, torch.float32):
        wrong = lambda x: wrong_outputs(x.to(dtype), o, scale, dk)  # noqa: E731
        assert wrong(o) == (0, 0)
        assert wrong(in_segments(tok, S0, lambda j, s: s)) == (0, 0)
        blocks = H * -(-T // 64)
        for x in (1.5 * o, torch.zeros_like(o), o.flip(1), (1 + 2.0 ** -6) * o):
            assert wrong(x)[1] == blocks
        # each of these is wrong in every block that begins a segment but the first
        begin = H * (-(-T // SEG) - 1)
        assert wrong(in_segments(tok, S0, lambda j, s: torch.zeros_like(s) if j else s))[1] >= begin
        assert wrong(in_segments(tok, S0, lambda j, s: s.flip(0) if j else s))[1] >= begin
        assert wrong(in_segments(tok, S0, lambda j, s: S0 if j else s))[1] >= begin
        one = o.clone()
        one[1000, 1] = 0
        assert wrong(one)[0] > 0
        assert wrong(torch.where(torch.arange(T)[:, None, None] == 77, float("nan"), o))[1] == H
    assert state_off(S.float(), S, dk) == 0
    assert state_off((S * (1 + 2.0 ** -16)).float(), S, dk) == H
    assert state_off(S.flip(0).float(), S, dk) == H


def test_a_float32_recurrence_is_within_the_noise():
    """The recurrence with every operation in 32 bits, outputs kept in 32 bits."""
    *tok, S0 = tokens(128, 128, 0.001)
    o, S64, scale = rule(*tok, S0)
    q, k, v, al, be = (x.float() for x in tok)
    S, got = S0.clone(), torch.empty_like(v)
    for t in range(T):
        S = S * al[t][:, None, None]
        u = be[t][:, None, None] * (v[t][:, None] - (S * k[t][:, :, None]).sum(1, keepdim=True))
        S = S + k[t][:, :, None] * u
        got[t] = (S * q[t][:, :, None]).sum(1)
    assert wrong_outputs(got, o, scale, 128) == (0, 0)
    assert state_off(S, S64, 128) == 0
