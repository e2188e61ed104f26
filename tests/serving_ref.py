"""Plain 64-bit references of the prompt, state-cache and output-norm calls
(test infrastructure, no code of the package)."""
import numpy as np


def delta_rule(q, k, v, alpha, beta, S):
    """One prompt, one head, token by token.  q, k [T, dk]; v [T, dv]; S
    [dk, dv].  Returns o [T, dv], the final state, and the largest column norm
    that any state had."""
    S = S.astype(np.float64).copy()
    o = np.zeros((len(q), v.shape[1]))
    top = np.sqrt((S ** 2).sum(0)).max() if S.size else 0.0
    for t in range(len(q)):
        u = beta[t] * (v[t] - alpha[t] * (S.T @ k[t]))
        S = alpha[t] * S + np.outer(k[t], u)
        o[t] = S.T @ q[t]
        top = max(top, np.sqrt((S ** 2).sum(0)).max())
    return o, S, top


def quantise(S, bits):
    """codes (int) and scales of a state [..., dv]; 32 values share a scale."""
    x = S.astype(np.float64).reshape(*S.shape[:-1], -1, 32)
    amax = np.abs(x).max(-1, keepdims=True)
    s = (amax / (127 if bits == 8 else 7)).astype(np.float32)
    finite = np.isfinite(amax)
    live = finite & (amax >= 2.0 ** -100)
    c = np.rint(np.divide(x, s.astype(np.float64), where=live, out=np.zeros_like(x)))
    s = np.where(live, s, np.where(finite, np.float32(0), np.float32(np.nan)))
    return np.where(live, c, 0).astype(np.int64).reshape(S.shape), s[..., 0]


def dequantise(codes, scale):
    """fp32 values, one rounding of code * scale."""
    x = codes.reshape(*codes.shape[:-1], -1, 32).astype(np.float32) * scale[..., None].astype(np.float32)
    return x.reshape(codes.shape)


def unpack4(packed):
    """[..., dv / 2] uint8 -> [..., dv] codes."""
    lo, hi = packed.astype(np.int64) & 15, packed.astype(np.int64) >> 4
    c = np.stack([lo, hi], -1).reshape(*packed.shape[:-1], -1)
    return np.where(c > 7, c - 16, c)


def _act(z, act):
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s if act == "silu" else s if act == "sigmoid" else z


def group_norm(x, weight, bias, gate, eps, act, centred, gate_first):
    x = x.astype(np.float64)
    if gate is not None and gate_first:
        x = x * _act(gate.astype(np.float64), act)
    mean = x.mean(-1, keepdims=True) if centred else 0.0
    y = (x - mean) / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    if gate is None:
        return _act(y, act)
    return y if gate_first else y * _act(gate.astype(np.float64), act)
