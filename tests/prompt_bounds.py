"""The delta rule in 64 bits with the scale of what fp32 arithmetic may be off
by, and bounds of a prompt's outputs that do not grow with its length (test
infrastructure, no code of the package)."""
import torch

EPS32 = 2.0 ** -24
BLOCK = 64


def rule(q, k, v, alpha, beta, S):
    """One prompt, all heads, token by token.  q, k [T, H, dk]; v [T, H, dv];
    alpha, beta [T, H]; S [H, dk, dv].  Returns o [T, H, dv], the final state and
    the scale [T, H, dv] of an output: |q_t| times the norm of the column of the
    state that it is read from."""
    q, k, v, alpha, beta = (x.double() for x in (q, k, v, alpha, beta))
    S = S.double().clone()
    o, scale = torch.empty_like(v), torch.empty_like(v)
    qn = q.norm(dim=-1)
    for t in range(len(q)):
        kt = k[t][:, :, None]
        S = S * alpha[t][:, None, None]
        u = beta[t][:, None, None] * (v[t][:, None] - (S * kt).sum(1, keepdim=True))
        S = S + kt * u
        o[t] = (S * q[t][:, :, None]).sum(1)
        scale[t] = qn[t][:, None] * S.norm(dim=1)
    return o, S, scale


def wrong_outputs(got, o, scale, dk):
    """How many outputs, and how many blocks of 64 tokens of a head, are off by
    more than half a step of their type and the noise of fp32 sums.

    The noise: an output is a sum of dk products, each rounded to 2^-24 of it, of
    a state column whose own error does not grow with the prompt: a token puts
    in at most a few roundings of 2^-24 of the column, of random signs, and keys
    and decays take away about beta / dk of what is in, so that the roundings of
    some dk tokens are what is there: sqrt(dk) 2^-24 of the column's norm, a few
    times.  Eight times is allowed for a block's norm, sixteen for one value
    (the largest of millions)."""
    half = torch.finfo(got.dtype).eps / 2
    d, o = (got.double() - o).abs(), o.abs()
    noise = dk ** 0.5 * EPS32 * scale
    ones = int((~(d <= half * o + 16 * noise)).sum())
    pad = -len(d) % BLOCK

    def norms(x):
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad))
        return x.reshape(-1, BLOCK, *x.shape[1:]).pow(2).sum((1, 3)).sqrt()

    blocks = int((~(norms(d) <= half * norms(o) + 8 * norms(noise))).sum())
    return ones, blocks


def state_off(got, S, dk):
    """Heads whose state is off by more than eight times the noise of its norm."""
    d = (got.double() - S).flatten(1).norm(dim=1)
    return int((~(d <= 8 * dk ** 0.5 * EPS32 * S.flatten(1).norm(dim=1))).sum())
