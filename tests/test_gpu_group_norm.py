"""The output group norm on the GPU against 64-bit arithmetic."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.serving import OutputNorm, group_norm

WIDTHS = [8, 16, 24, 40, 64, 128, 200, 256, 504, 512, 520, 1024, 1032, 2048, 2056, 4096, 5000, 8192]


def data(rows, groups, width, dt, seed, offset=0.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, groups * width + pad), generator=g, device="cuda") * 2 + offset
    return x.to(dt)[:, :groups * width].unflatten(1, (groups, width))


def check(x, y, norm, gate, rows=None):
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want = ref.group_norm(f(x), f(norm.weight), f(norm.bias), f(gate), norm.eps, norm.act, norm.centred, norm.gate_first)
    got = f(y)
    W = x.shape[-1]
    # fp32: the sums of W terms (in partial sums of at most 64 terms a lane, joined
    # over at most 256 lanes) relative to the group's norm, a dozen roundings of the
    # result, the exponential's 2^-22 times its argument; then half a step of y
    mag = np.abs(want) + np.sqrt((want ** 2).mean(-1, keepdims=True)) + (0 if norm.bias is None else np.abs(f(norm.bias)))
    big = 0.0
    for z in (f(gate), want if gate is None else None):
        big = max(big, 0.0 if z is None else np.abs(z[np.isfinite(z)]).max(initial=0.0))
    e32 = (np.sqrt(W) + 32 + 4 * big) * 2.0 ** -24
    if norm.centred:
        xx = f(x)
        m = np.abs(xx.mean(-1, keepdims=True)) / np.sqrt(xx.var(-1, keepdims=True) + norm.eps)
        mag = mag + (np.sqrt(W) + 8) * m       # the mean's own roundings, over the deviation
    half = torch.finfo(y.dtype).eps / 2
    lim = half * np.abs(want) + e32 * mag * (1 if norm.weight is None else 1 + np.abs(f(norm.weight)).max())
    assert (np.abs(got - want) <= lim * (1 + half)).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dt):
    for rows, groups in ((1, 1), (3, 5), (37, 3)):
        x, z = data(rows, groups, width, dt, 1), data(rows, groups, width, dt, 2)
        y = torch.full_like(x, 9.0)
        norm = OutputNorm(1 + 0.3 * torch.randn(groups, width, device="cuda"))
        assert group_norm(x, norm, y, gate=z) == 0
        check(x, y, norm, z)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("gate", ["none", "first", "after"])
def test_forms(dt, act, centred, gate):
    for width in (64, 1032, 2056):
        rows, groups = 19, 2
        x = data(rows, groups, width, dt, 3, offset=1.0, pad=16)
        z = None if gate == "none" else data(rows, groups, width, dt, 4, pad=32)
        shared = gate == "after"
        w = 1 + 0.3 * torch.randn((width,) if shared else (groups, width), device="cuda")
        b = 0.2 * torch.randn_like(w) if centred else None
        norm = OutputNorm(w, b, 1e-6, act, centred, gate == "first")
        y = torch.full((rows, groups * width + 48), 5.0, device="cuda", dtype=dt)
        yv = y[:, :groups * width].unflatten(1, (groups, width))
        assert group_norm(x, norm, yv, gate=z) == 0
        check(x, yv, norm, z)
        assert (y[:, groups * width:] == 5).all()


def test_many_rows_in_place_and_on_another_stream():
    x = data(20011, 4, 128, torch.bfloat16, 5)
    z = data(20011, 4, 128, torch.bfloat16, 6)
    norm = OutputNorm(torch.rand(128, device="cuda"))
    y = x.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert group_norm(y, norm, y, gate=z) == 0
    torch.cuda.synchronize()
    check(x, y, norm, z)
    assert group_norm(x, norm, z, gate=z) == 0           # over the gate
    torch.cuda.synchronize()
    assert torch.equal(z, y)


def test_zero_rows_constant_groups_and_non_finite_values():
    norm = OutputNorm(eps=1e-5)
    x = torch.zeros((4, 2, 64), device="cuda")
    y = torch.empty_like(x)
    assert group_norm(x[:0], norm, y[:0]) == 0
    assert group_norm(x, OutputNorm(act="none"), y) == 0
    assert not y.any()
    x[1] = 1e4
    assert group_norm(x, OutputNorm(act="none", centred=True), y) == 0
    assert not y.any()                                   # a group that is all one value
    x.normal_()
    x[2, 1, 5] = float("nan")
    x[3, 0, 9] = float("inf")
    assert group_norm(x, OutputNorm(act="none"), y) == 0
    assert y[2, 1].isnan().all() and y[2, 0].isfinite().all() and y[:2].isfinite().all() and y[3, 1].isfinite().all()
    z = torch.zeros_like(x)
    z[0, 0, :3] = torch.tensor([-1e4, 1e4, -200.0])      # where exp over- and underflows
    x = torch.ones_like(x)
    assert group_norm(x, OutputNorm(act="sigmoid", eps=0.0), y, gate=z) == 0
    assert y[0, 0, :4].tolist() == [0.0, 1.0, 0.0, 0.5]


def test_graph_replays():
    x, z = data(300, 3, 64, torch.bfloat16, 7), data(300, 3, 64, torch.bfloat16, 8)
    norm, y = OutputNorm(torch.rand(3, 64, device="cuda")), torch.empty_like(x)
    group_norm(x, norm, y, gate=z)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert group_norm(x, norm, y, gate=z) == 0
    for rep in range(3):
        x.copy_(data(300, 3, 64, torch.bfloat16, 20 + rep))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(x, y, norm, z)


@pytest.mark.parametrize("lo,hi", [(0, 40), (3, 37), (7, 8), (5, 5), (20, 10), (-4, 12), (30, 900), (-9, -2), (41, 50)])
def test_part_of_the_rows(lo, hi):
    """Rows from the first up to the last entry of a device list, within [0, rows);
    the others are left as they were, in place too."""
    for width in (64, 2056):
        x = data(40, 3, width, torch.bfloat16, 4)
        rows = torch.tensor([lo, 17, hi], dtype=torch.int32, device="cuda")
        norm, y = OutputNorm(None, act="none"), x.clone()
        assert group_norm(y, norm, y, rows=rows) == 0
        a, b = max(lo, 0), min(hi, 40)
        inside = slice(a, max(a, b))
        check(x[inside], y[inside], norm, None)
        out = torch.ones(40, dtype=torch.bool)
        out[inside] = False
        assert torch.equal(y[out], x[out])


@pytest.mark.parametrize("dt,rows,groups,width", [(torch.bfloat16, 16387, 8, 136), (torch.float32, 700, 3, 4104)])
def test_outputs_beyond_the_caches(dt, rows, groups, width):
    """More than 32 MiB of output, in place, with every row's neighbours at a stride."""
    x = data(rows, groups, width, dt, 5, pad=8)
    norm, whole = OutputNorm(None, torch.full((width,), 0.5, device="cuda"), act="none"), x.clone()
    store = torch.full((rows, groups * width + 8), 3.0, device="cuda", dtype=dt)
    y = store[:, :groups * width].unflatten(1, (groups, width))
    y.copy_(x)
    assert rows * groups * width * x.element_size() > 32 << 20
    assert group_norm(y, norm, y) == 0
    check(whole, y, norm, None)
    assert (store[:, groups * width:] == 3).all()
