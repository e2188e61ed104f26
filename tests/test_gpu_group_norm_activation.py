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
    exponential instruction two (one unit in the last place), its correction's
    rounding one, the sum with one, its reciprocal and each of two products one:
    seven; an exponential under the normal range may be lost (x times 2^-126).  bf16: half a step and 2^-22 (1 + |z|) of
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
    units = 7 if form != "first" else 11
    if dt == torch.float32:
        lim = units * 2.0 ** -24 * want.abs() + (1 + w.abs()) * 2.0 ** -126
    else:
        lim = (2.0 ** -8 + 2.0 ** -22 * (1 + w.abs()) + units * 2.0 ** -24) * want.abs() + 2.0 ** -118
    assert ((y.double() - want).abs() <= lim).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_activations_of_what_is_no_finite_number(dt):
    inf, nan, top = float("inf"), float("nan"), torch.finfo(dt).max
    z = torch.tensor([inf, -inf, nan, top, -top, 0.0, -0.0, 128.5], device="cuda").to(dt).repeat(3, 1, 8)
    one, y = torch.ones_like(z), torch.empty_like(z)
    assert group_norm(one, OutputNorm(eps=0.0, act="sigmoid"), y, gate=z) == 0
    want = torch.tensor([1, 0, nan, 1, 0, 0.5, 0.5, 1], device="cuda").to(dt).repeat(3, 1, 8)
    assert torch.equal(y.nan_to_num(7), want.nan_to_num(7))
    assert group_norm(one, OutputNorm(eps=0.0, act="silu"), y, gate=z) == 0
    assert y[0, 0, :8].tolist()[0] == inf and y[0, 0, 2].isnan() and y[0, 0, 3] == z[0, 0, 3] and y[0, 0, 4] == 0
    assert y[0, 0, 5] == 0 and y[0, 0, 7] == z[0, 0, 7] and y[0, 0, 1].isnan()          # (-inf / inf)
