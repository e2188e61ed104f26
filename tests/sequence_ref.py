"""Plain 64-bit references of the scan, convolution and beam calls, with the bounds
that fp32 arithmetic keeps (test infrastructure, no code of the package)."""
import numpy as np

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}       # half a step, relative
U = 2.0 ** -24


def scan(q, k, v, dt, A, S):
    """One prompt, token by token.  q, k [T, G, dk]; v [T, H, dv]; dt [T, H]; A
    [H]; S [H, dk, dv].  Returns o [T, H, dv], the final state, and how far fp32
    sums may be off both: M is the state with every term's magnitude, E the sum
    of every term times the magnitude of its decays' logarithms.  A term takes
    from each later token two roundings of the decay and one or two of a sum,
    three more where an operand enters as three values (at most 8 a token), and
    four units of the logarithm's own value; an output's sum over dk products, of
    three values each, takes 4 dk."""
    H, E_ = v.shape[1], v.shape[1] // k.shape[1]
    S = S.astype(np.float64).copy()
    M, E = np.abs(S), np.zeros_like(S)
    o, off = np.zeros(v.shape), np.zeros(v.shape)
    rate = np.exp(A.astype(np.float64))
    n = np.zeros(H)
    for t in range(len(v)):
        kk, qq = np.repeat(k[t], E_, 0), np.repeat(q[t], E_, 0)
        l = (dt[t] * rate)[:, None, None]
        a = np.exp(-l)
        term = dt[t][:, None, None] * kk[:, :, None] * v[t][:, None, :]
        E = a * (E + l * M)
        S, M = a * S + term, a * M + np.abs(term)
        n = n + 8
        o[t] = (qq[:, :, None] * S).sum(1)
        aq = np.abs(qq)[:, :, None]
        off[t] = U * ((n[:, None] + 4 * k.shape[2] + 8) * (aq * M).sum(1) + 4 * (aq * E).sum(1))
    return o, S, off, U * ((n[:, None, None] + 8) * M + 4 * E)


def sketch(S, P, off):
    """U rows of one sequence and how far an fp32 sum of the fp32 state may be off."""
    rows, tol = [], []
    for h in range(len(off) - 1):
        for j in range(off[h], off[h + 1]):
            rows.append((P[j][:, None] * S[h]).sum(0))
            tol.append(S.shape[1] * U * (np.abs(P[j])[:, None] * np.abs(S[h])).sum(0))
    return (np.stack(rows), np.stack(tol)) if rows else (np.zeros((0, S.shape[2])), np.zeros((0, S.shape[2])))


def silu(y):
    return y / (1.0 + np.exp(-y))


def conv(x, held, w, b, act):
    """One prompt: x [T, C], held [taps - 1, C], w [C, taps].  Returns y in front of
    and behind the activation, the sums' magnitudes and the new held inputs."""
    rows, taps, T = np.concatenate([held, x]), w.shape[1], len(x)
    y, m = np.zeros((T, x.shape[1])) + b, np.zeros((T, x.shape[1])) + np.abs(b)
    for j in range(taps):
        y, m = y + rows[j:j + T] * w[:, j], m + np.abs(rows[j:j + T] * w[:, j])
    out = silu(y) if act == "silu" else 1 / (1 + np.exp(-y)) if act == "sigmoid" else y
    return y, out, m, rows[T:]


def beams(x, scores, ended, end):
    """x [n, k, V]: the best k of every group, by score and then by index."""
    n, k, V = x.shape
    x = x.astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        top = x.max(-1, keepdims=True)
        lse = np.where(np.isfinite(top), top, 0) + np.log(np.exp(x - np.where(np.isfinite(top), top, 0)).sum(-1, keepdims=True))
        c = scores.astype(np.float64)[..., None] + (x - np.where(np.isfinite(lse), lse, 0))
    c[np.isneginf(scores)] = -np.inf
    over = (ended != 0)
    c[over] = -np.inf
    for g, b in zip(*np.nonzero(over)):
        c[g, b, max(end, 0)] = scores[g, b]
    c = c.reshape(n, k * V)
    parents, tokens, out, done = (np.zeros((n, k), d) for d in (np.int64, np.int64, np.float64, np.int64))
    for g in range(n):
        order = np.lexsort((np.arange(k * V), -c[g]))[:k]
        for r in range(k):
            at = order[r] if r < len(order) else 0
            if r >= len(order) or np.isneginf(c[g, at]):
                parents[g, r], tokens[g, r], out[g, r] = g * k + r, -1, -np.inf
                continue
            b = at // V
            parents[g, r], out[g, r] = g * k + b, c[g, at]
            tokens[g, r] = end if over[g, b] else at % V
            done[g, r] = over[g, b] or tokens[g, r] == end
    return parents, tokens, out, done
