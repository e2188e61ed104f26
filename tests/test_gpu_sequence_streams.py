"""Scans, convolutions, beam selections and reorderings on other streams than their
tensors': objects dropped while a call still uses them, two calls at once, and
offsets past 2^32."""
import numpy as np
import pytest
import torch

from tests import test_gpu_beams as beams
from tests import test_gpu_conv as conv
from tests import test_gpu_scan as scan
from tests.test_gpu_serving_streams import BUSY, reused

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.layer import DecodeLayer
    from ssm_decode_amd.serving import BeamSearch, ScanPrompts


def busy():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    return side


@pytest.mark.parametrize("given", ["handle", "current"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_prompts_dropped_behind_their_scan(act, given):
    lens = [1300]                                # (in segments: the workspace counts)
    lay = scan.make_layer(1, 4, 2, 128, 64, act, seed=500)
    tok = scan.make_tokens(1300, 4, 2, 128, 64, act, seed=501)
    S0 = scan.f64(lay.S)
    pr = ScanPrompts(lay, *tok, scan.ints(scan.starts(lens)))
    at, size = {pr.work.data_ptr(), pr.seq_start.data_ptr()}, [pr.work.numel(), 8]
    assert pr.work.numel() > 0
    side = busy()
    if given == "handle":
        assert lay.scan(pr, stream=side.cuda_stream) == 0
    else:
        with torch.cuda.stream(side):
            assert lay.scan(pr) == 0
    del pr
    assert not side.query()
    assert not reused(at, size)
    assert not side.query()
    torch.cuda.synchronize()
    scan.check(lay, tok, lens, [0], [1], S0)


def test_a_convolution_dropped_behind_its_call():
    c = conv.Case(5, 5, seed=502)
    lay, taps = c.lay, c.conv.taps
    at = {c.conv.state.data_ptr(), c.conv.weight.data_ptr(), c.conv.bias.data_ptr()}
    size = [c.conv.state.numel() * 2, c.conv.weight.numel() * 4, c.conv.bias.numel() * 4]
    w, b, held = c.conv.weight.double(), c.conv.bias.double(), c.held.double()
    side = busy()
    assert c.call(stream=side.cuda_stream) == 0
    c.conv = None
    assert not side.query()
    assert not reused(at, size)
    assert not side.query()
    torch.cuda.synchronize()
    x = torch.cat([held, c.x.double()[:, None]], 1)
    z = b + (x * w.t()[None]).sum(1)
    m = b.abs() + (x.abs() * w.t()[None].abs()).sum(1)
    y = z / (1 + torch.exp(-z))
    # the class's tolerance: taps + 1 roundings of the terms, the activation's units, one to bf16
    tol = 2.0 ** -8 * y.abs() + 1.01 * 2.0 ** -24 * (1.1 * (taps + 1) * m + (16 + 2 * z.abs()) * y.abs())
    assert ((c.y[:, :y.shape[1]].double() - y).abs() <= tol).all()
    assert lay.error_word() == 0


def test_a_search_dropped_behind_its_selection():
    n, k, V = 3, 4, 20011
    x, s = beams.inputs(n, k, V, "bf16", seed=503)
    search, want = BeamSearch(n, k, V), BeamSearch(n, k, V)
    e = torch.zeros_like(search.ended)
    assert want.select(x, s, e) == 0
    at, size = {search.work.data_ptr()}, [search.work.numel() * search.work.element_size()]
    out = search.parents, search.tokens, search.scores, search.ended
    side = busy()
    assert search.select(x, s, e, stream=side.cuda_stream) == 0
    del search
    assert not side.query()
    assert not reused(at, size)
    assert not side.query()
    torch.cuda.synchronize()
    beams.check(want, x, s, e)
    for a, b in zip(out, (want.parents, want.tokens, want.scores, want.ended)):
        assert torch.equal(a, b)


def test_a_convolution_dropped_behind_its_reordering():
    lay, cv, held = beams.make("mamba2", 24, H=64, G=4, dk=128, dv=128, W=4, act="bf16", seed=504)
    at = torch.tensor([b // 3 * 3 + (2 * b + b // 3) % 3 for b in range(24)], dtype=torch.int32, device="cuda")
    place, size = cv.state.data_ptr(), cv.state.numel() * 2
    held = {n: x for n, x in held.items() if x.data_ptr() != place}
    want = {n: x[at.long()].clone() for n, x in held.items()}
    side = busy()
    assert lay.reorder(at, 3, convs=(cv,), stream=side.cuda_stream) == 0
    del cv
    assert not side.query()
    assert not reused({place}, [size])
    assert not side.query()
    torch.cuda.synchronize()
    for n, x in held.items():
        assert torch.equal(x, want[n]), n


def test_two_convolutions_at_once():
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    at = [0, 200, 201, 300]
    cases = [conv.Case(300, 3, seed=510 + n, unit=True, fn="silu") for n in range(2)]
    st = conv.ints(at)
    torch.cuda.synchronize()
    for s in side:
        with torch.cuda.stream(s):
            torch.cuda._sleep(1 << 24)
    for s, c in zip(side, cases):
        assert c.call(seq_start=st, stream=s.cuda_stream) == 0
    torch.cuda.synchronize()
    for c in cases:
        c.check(at, [0, 1, 2], [1, 1, 1])


def test_two_selections_at_once():
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    n, k, V = 4, 5, 30000
    made = [(BeamSearch(n, k, V), *beams.inputs(n, k, V, "bf16", seed=520 + i)) for i in range(2)]
    e = torch.zeros((n, k), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for s in side:
        with torch.cuda.stream(s):
            torch.cuda._sleep(1 << 24)
    for s, (search, x, sc) in zip(side, made):
        assert search.select(x, sc, e, stream=s.cuda_stream) == 0
    torch.cuda.synchronize()
    for search, x, sc in made:
        beams.check(search, x, sc, e)


# ------------------------------------------------------ offsets past 2^32
def test_states_past_2_32_bytes_move():
    B, H = 1200, 64                              # (4 MiB a sequence: 4.7 GiB)
    lay = DecodeLayer("mamba2", B, H, 4, 128, 128, 4, "bf16", "bf16", np.arange(H + 1) * 2)
    g = torch.Generator(device="cuda").manual_seed(530)
    mark = torch.randn((H, 128, 128), generator=g, device="cuda")
    for b in (0, 1, B - 4, B - 3, B - 2, B - 1):
        lay.S[b] = mark + b
    at = torch.arange(B, dtype=torch.int32, device="cuda")
    at[:4] = torch.tensor([1, 1, 2, 3])
    at[-4:] = B - 4 + torch.tensor([3, 0, 2, 0])
    assert lay.reorder(at, 4) == 0
    for b, p in ((0, 1), (1, 1), (B - 4, B - 1), (B - 3, B - 4), (B - 2, B - 2), (B - 1, B - 4)):
        assert torch.equal(lay.S[b], mark + p), b
    assert lay.error_word() == 0


@pytest.mark.parametrize("step", [False, True])
def test_convolution_rows_far_apart(step):
    N = 80
    c = conv.Case(N, N if step else 1, H=1, G=1, dk=64, dv=64, seed=531)
    wide = 1 << 25                               # (64 MiB a row: rows from the 65th on lie past 2^32 bytes)
    far = torch.empty(wide * (N - 1) + 512, dtype=torch.bfloat16, device="cuda")
    x = far.as_strided((N, 192), (wide, 1), 0)
    x.copy_(c.x)
    c.x = x
    near, c.y = c.y, far.as_strided((N, c.y.shape[1]), (wide, 1), 192)
    c.y.copy_(near)
    first, out = 0, {}
    for n in c.order:
        out[n] = far.as_strided((N, 1, 64), (wide, 64, 1), 192 + first)
        first += 64
    c.out = out
    if step:
        assert c.call() == 0
        c.check(list(range(N + 1)), list(range(N)), [1] * N)
    else:
        assert c.call(seq_start=conv.ints([0, N])) == 0
        c.check([0, N], [0], [1])
