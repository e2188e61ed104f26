"""The norm's activations alone: groups of ones have themselves as norm."""
import pytest
import torch

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.serving import OutputNorm, group_norm


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("form", ["after", "first", "none"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_activations_over_their_range(act, form, dt):
    """With eps = 0 a group of ones is its norm, exactly (the sum of 64 ones, its
    mean, one over its root).  fp32, in units of 2^-24 of the result: the
    exponential within two (one unit in the last place), one for the sum with
    one, one for the quotient, one for each of two products: six; results under the normal
    range may be lost to it (x times 2^-126).  bf16: half a step and 2^-22 (1 + |z|) of
    the result, and what is under 2^-118 may become 0."""
    z = torch.linspace(-100, 100, 64 * 4001, device="cuda").reshape(-1, 1, 64).to(dt)
    one = torch.ones_like(z)
    y = torch.empty_like(z)
    if form == "after":
        norm, args = OutputNorm(eps=0.0, act=act), (one, z)
    elif form == "none":                     # the result's own activation: the bias is the argument
        norm, args = None, (one, None)
    else:                                    # beside this eps the mean of squares is nothing
        norm, args = OutputNorm(eps=1e30, act=act, gate_first=True), (one, z)
    w = z.double()
    want = 1 / (1 + torch.exp(-w)) * (w if act == "silu" else 1)
    if form == "none":                       # one row a call: weight 0, the arguments as bias
        rows = torch.linspace(0, 4000, 41).long().tolist()
        for r in rows:
            n = OutputNorm(torch.zeros(1, 64, device="cuda"), z[r].float().contiguous(), eps=0.0, act=act)
            assert group_norm(one[r:r + 1], n, y[r:r + 1]) == 0
        y, want, w = y[rows], want[rows], w[rows]
    else:
        assert group_norm(args[0], norm, y, gate=args[1]) == 0
        if form == "first":                  # x' / sqrt(mean + eps)
            want = want / torch.sqrt((want * want).mean(-1, keepdim=True) + float(torch.tensor(1e30, dtype=torch.float32)))
    # (first: a sum, a root, a reciprocal and a product more)
    units = 6 if form != "first" else 10
    if dt == torch.float32:
        lim = units * 2.0 ** -24 * want.abs() + (1 + w.abs()) * 2.0 ** -126
    else:
        lim = (2.0 ** -8 + 2.0 ** -22 * (1 + w.abs()) + units * 2.0 ** -24) * want.abs() + 2.0 ** -118
    assert ((y.double() - want).abs() <= lim).all()
