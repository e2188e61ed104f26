"""Chunks whose factors dt (q . k) are large and whose values are small: every term is far
from the type's end, and so are the outputs (tolerances: tests/sequence_ref.py)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_scan import check, f64, ints, make_layer, make_tokens, starts

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.serving import ScanPrompts


@pytest.mark.parametrize("H,G,dk,dv", [(4, 2, 128, 64), (16, 1, 64, 64), (5, 1, 128, 128)])
@pytest.mark.parametrize("qk,dt,rows", [(52, 0.4, slice(0, 200)), (52, 0.4, slice(110, 120)), (52, 0.4, slice(126, 130)), (36, 2.0 ** 30, slice(0, 200)),
                                        (36, 2.0 ** 30, slice(60, 61))])
def test_large_factors_of_small_values(H, G, dk, dv, qk, dt, rows):
    """q and k of 2^qk in some rows, decays of 2^-37 a chunk: dt (q . k) over a chunk's first
    decays passes 2^128, its terms with v of 2^-60 stay under 2^50."""
    lens = [200, 90]
    lay = make_layer(2, H, G, dk, dv, "bf16", seed=700)
    q, k, v, d, o = make_tokens(sum(lens), H, G, dk, dv, "bf16", seed=701)
    d.fill_(dt)
    lay.A.fill_(float(np.log(0.4 / dt)))
    lay.S.mul_(2.0 ** -40)
    v.mul_(2.0 ** -60)
    q[rows] *= 2.0 ** qk
    k[rows] *= 2.0 ** qk
    S0 = f64(lay.S)
    assert lay.scan(ScanPrompts(lay, q, k, v, d, o, ints(starts(lens)))) == 0
    assert np.isfinite(f64(o)).all() and np.isfinite(f64(lay.S)).all()
    check(lay, (q, k, v, d, o), lens, [0, 1], [1, 1], S0)
