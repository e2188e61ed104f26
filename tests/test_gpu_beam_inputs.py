"""The inputs of tests/test_gpu_beams.py decide their parents: where neighbouring
candidates of a group are of different beams, their scores are further apart than the
sums' errors can bring them (candidates of one beam are ordered by value, which no sum enters).

A beam's logarithm of V exponentials in fp32 is off by its sum's relative error: an
exponential by 2^-23 of itself, for the instruction, and 2^-24 of its exponent's magnitude a times it
(a e^-a is under a half: 2^-25 of the largest term, and of the sum); a lane's 32 values one
after the other 32 roundings, the wave's tree 6; 64 bits behind that.  Together under 42 of 2^-24;
two beams' differ by at most twice that."""
import numpy as np
import pytest

from tests import test_gpu_beams as beams

pytestmark = pytest.mark.gpu
APART = 2 * 42 * 2.0 ** -24


def closest(x, scores, ended, end):
    """The least distance of two neighbours of different beams among the best and the one behind them."""
    n, k, V = x.shape
    least = np.inf
    for g in range(n):
        cand = []
        for b in range(k):
            if np.isneginf(scores[g, b]):
                continue
            if ended[g, b]:
                cand.append((scores[g, b], b))
                continue
            row = x[g, b][np.isfinite(x[g, b])]
            if len(row) == 0:
                continue
            top = row.max()
            lse = top + np.log(np.exp(row - top).sum())
            best = np.sort(row)[::-1][:k + 1]
            cand += [(scores[g, b] + (v - lse), b) for v in best]
        cand.sort(key=lambda c: -c[0])
        for (s, a), (t, b) in zip(cand[:k + 1], cand[1:k + 1]):
            if a != b:
                least = min(least, s - t)
    return least


def marks(f):
    """Every combination of a test's parameters."""
    out = [{}]
    for m in getattr(f, "pytestmark", []):
        if m.name == "parametrize":
            names = [n.strip() for n in m.args[0].split(",")]
            out = [dict(o, **dict(zip(names, v if len(names) > 1 else (v,)))) for o in out for v in m.args[1]]
    return out


@pytest.mark.parametrize("name", ["test_selection", "test_a_first_step_has_one_beam", "test_ended_beams_and_ruled_out_tokens",
                                  "test_wrong_logits_take_their_beam_out", "test_captured_and_replayed", "test_rows_far_apart"])
def test_candidates_are_apart(name, monkeypatch):
    seen = []

    def check(search, x, scores, ended, err=0):
        n, k = scores.shape
        seen.append(closest(beams.f64(x).reshape(n, k, -1), beams.f64(scores), ended.cpu().numpy(), search.end))

    monkeypatch.setattr(beams, "check", check)
    for kw in marks(getattr(beams, name)):
        getattr(beams, name)(**kw)
        assert seen and min(seen) > APART, (kw, min(seen))
