"""The quantised state cache on the GPU against 64-bit arithmetic: codes and
scales bit for bit, what is read back, refusals, graphs, and decode steps that
go on from it."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd import abi
    from ssm_decode_amd.layer import DecodeLayer
    from ssm_decode_amd.serving import StateCache

SHAPES = [(16, 32), (64, 64), (128, 64), (128, 128)]


def make_layer(B, H, dk, dv, act="bf16", family="gdn", groups=None, seed=0, ranks=None):
    ranks = [(2 + 3 * h) % 9 for h in range(H)] if ranks is None else ranks
    off = np.concatenate([[0], np.cumsum(ranks)]).astype(np.int32)
    lay = DecodeLayer(family, B, H, groups or H, dk, dv, 4, act, act, off)
    g = torch.Generator(device="cuda").manual_seed(seed)
    lay.S.copy_(torch.randn(lay.S.shape, generator=g, device="cuda"))
    lay.Pt.copy_(torch.randn(lay.Pt.shape, generator=g, device="cuda") / dk ** 0.5)
    lay.Cmap.copy_(lay.Pt)
    return lay


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def codes_of(cache):
    c = cache.codes.cpu().numpy()
    return c.astype(np.int64) if cache.bits == 8 else ref.unpack4(c)


def check_slot(cache, slot, S):
    c, s = ref.quantise(S.cpu().numpy(), cache.bits)
    assert np.array_equal(codes_of(cache)[slot], c)
    assert np.array_equal(cache.scale[slot].cpu().numpy(), s, equal_nan=True)


def check_loaded(lay, b, cache, slot):
    want = ref.dequantise(codes_of(cache)[slot], cache.scale[slot].cpu().numpy())
    assert np.array_equal(lay.S[b].cpu().numpy(), want, equal_nan=True)
    off, P, dense = lay.offsets_host, lay.Pt.double().cpu().numpy(), {h: j for j, h in enumerate(lay.dense_heads)}
    half = torch.finfo(lay.U.dtype).eps / 2
    for h in range(lay.H):
        if h in dense:
            assert torch.equal(lay.Scopy[b, dense[h]], lay.S[b, h].to(lay.Scopy.dtype))
            continue
        r = slice(off[h], off[h + 1])
        U = P[r] @ want[h].astype(np.float64)
        # fp32 sums of dk terms, then one rounding to the sketch's type
        lim = half * np.abs(U) + (lay.dk + 2) * 2.0 ** -24 * (np.abs(P[r]) @ np.abs(want[h].astype(np.float64)))
        assert (np.abs(lay.U[b, r].double().cpu().numpy() - U) <= lim * (1 + half)).all()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("family,act", [("gdn", "bf16"), ("kda", "f32"), ("mamba2", "bf16")])
def test_round_trip(bits, dk, dv, family, act):
    H = 6
    lay = make_layer(7, H, dk, dv, act, family, 2 if family == "mamba2" else H, seed=dk + dv + bits)
    lay.S.mul_(torch.rand((7, H, dk, 1), device="cuda") * 3)
    cache = StateCache(lay, 5, bits)
    S0 = lay.S.clone()
    assert lay.save_state(cache, ints(6, 0, 3), ints(4, 1, 0)) == 0
    torch.cuda.synchronize()
    assert torch.equal(lay.S, S0)
    for b, slot in ((6, 4), (0, 1), (3, 0)):
        check_slot(cache, slot, S0[b])
    assert not cache.codes[2].any() and not cache.codes[3].any() and not cache.scale[2:4].any()
    lay.count.fill_(3)                                   # what was in the rings is dropped
    assert lay.load_state(cache, ints(2, 5, 1), ints(4, 4, 0)) == 0
    torch.cuda.synchronize()
    for b, slot in ((2, 4), (5, 4), (1, 0)):
        check_loaded(lay, b, cache, slot)
    assert lay.count.cpu().numpy()[:, 0].tolist() == [3, 0, 0, 3, 3, 0, 3]
    for b in (0, 3, 4, 6):
        assert torch.equal(lay.S[b], S0[b])
    assert lay.error_word() == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_values_at_the_borders_between_codes(bits):
    """Halves between two codes go to the even one, and their neighbours in
    fp32 to the nearest, at scales that divide nothing evenly."""
    top = 127 if bits == 8 else 7
    lay = make_layer(4, 2, 64, 64)
    x = np.zeros((4, 2, 64, 2, 32), np.float32)
    rng = np.random.default_rng(3)
    amax = np.exp2(rng.uniform(-90, 90, x.shape[:-1] + (1,))).astype(np.float32)
    amax[0] = top * np.exp2(rng.integers(-90, 90, amax[0].shape))      # scales that are powers of two
    s = (amax.astype(np.float64) / top).astype(np.float32)
    half = rng.integers(-top, top, x.shape) + 0.5
    x[:] = (half * s).astype(np.float32)
    step = rng.integers(-2, 3, x.shape)
    for n in (1, 2):
        x = np.where(np.abs(step) >= n, np.nextafter(x, np.where(step > 0, np.inf, -np.inf).astype(np.float32)), x)
    x[..., :1] = amax
    x = np.clip(x, -amax, amax).astype(np.float32).reshape(4, 2, 64, 64)
    lay.S.copy_(torch.from_numpy(x))
    cache = StateCache(lay, 4, bits)
    assert lay.save_state(cache, ints(0, 1, 2, 3), ints(0, 1, 2, 3)) == 0
    torch.cuda.synchronize()
    for b in range(4):
        check_slot(cache, b, lay.S[b])


@pytest.mark.parametrize("bits", [8, 4])
def test_zeros_tiny_huge_and_non_finite_blocks(bits):
    lay = make_layer(1, 2, 64, 64)
    S = lay.S[0]
    S[0, 0] = 0
    S[0, 1] = 2.0 ** -101
    S[0, 2] *= 2.0 ** -100
    S[0, 3, 0] = 2.0 ** -100
    S[0, 4] = 3.4e38
    S[0, 5, 7] = float("inf")
    S[0, 6, 40] = float("nan")
    S[0, 7, 3] = -float("inf")
    S[0, 8] = 1e-42
    cache = StateCache(lay, 1, bits)
    assert lay.save_state(cache, ints(0), ints(0)) == 0
    torch.cuda.synchronize()
    check_slot(cache, 0, S)
    assert lay.load_state(cache, ints(0), ints(0), prime=False) == 0
    torch.cuda.synchronize()
    got = lay.S[0]
    assert not got[0, 0].any() and not got[0, 1].any() and not got[0, 8].any()
    assert got[0, 5, :32].isnan().all() and got[0, 5, 32:].isfinite().all()
    assert got[0, 6, 32:].isnan().all() and got[0, 6, :32].isfinite().all()
    assert got[0, 7, :32].isnan().all() and got[0, 4].isfinite().all()
    assert got[1].isfinite().all()


def test_refused_entries():
    lay = make_layer(6, 3, 64, 64)
    cache = StateCache(lay, 3)
    S0 = lay.S.clone()
    lay.count[2] = 1
    assert lay.save_state(cache, ints(0, 6, -1), ints(0, 1, 2)) == 0
    assert lay.error_word() == abi.SKSSM_ERRBIT_SEQ
    lay.err.zero_()
    assert lay.save_state(cache, ints(2), ints(1)) == 0
    assert lay.error_word() == abi.SKSSM_ERRBIT_COUNT
    lay.err.zero_()
    assert lay.save_state(cache, ints(1, 3, 4, 5), ints(2, 3, -1, 2)) == 0    # slot 2 twice: the first is taken
    assert lay.error_word() == abi.SKSSM_ERRBIT_SLOT
    check_slot(cache, 0, S0[0])
    check_slot(cache, 2, S0[1])
    assert not cache.codes[1].any()
    lay.err.zero_()
    assert lay.load_state(cache, ints(3, 3, 4, 9), ints(0, 2, 3, 0)) == 0     # sequence 3 twice
    torch.cuda.synchronize()
    assert lay.error_word() == abi.SKSSM_ERRBIT_SEQ | abi.SKSSM_ERRBIT_SLOT
    check_loaded(lay, 3, cache, 0)
    for b in (0, 1, 2, 4, 5):
        assert torch.equal(lay.S[b], S0[b])
    assert lay.save_state(cache, ints(), ints()) == 0 and lay.load_state(cache, ints(), ints()) == 0


def test_dense_heads_without_priming_and_f32_copies():
    lay = make_layer(2, 3, 128, 64, "f32", ranks=[0, 5, 0])
    cache = StateCache(lay, 1, 8)
    U0, C0 = lay.U.clone(), lay.Scopy.clone()
    lay.save_state(cache, ints(0), ints(0))
    lay.load_state(cache, ints(1), ints(0), prime=False)
    torch.cuda.synchronize()
    assert torch.equal(lay.U, U0) and torch.equal(lay.Scopy, C0)
    lay.load_state(cache, ints(1), ints(0))
    torch.cuda.synchronize()
    check_loaded(lay, 1, cache, 0)


def test_graph_replays_and_another_stream():
    lay = make_layer(4, 4, 128, 128, seed=9)
    cache = StateCache(lay, 2, 8)
    seqs, slots, dst = ints(0, 1), ints(1, 0), ints(2, 3)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lay.save_state(cache, seqs, slots)
        lay.load_state(cache, dst, slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert lay.save_state(cache, seqs, slots) == 0
        assert lay.load_state(cache, dst, slots) == 0
    for rep in range(4):
        lay.S.normal_()
        seqs.copy_(ints(rep % 2, 1 - rep % 2))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            check_slot(cache, int(slots[i]), lay.S[int(seqs[i])])
            check_loaded(lay, int(dst[i]), cache, int(slots[i]))


def test_restored_sequence_decodes_on():
    """A window of reads and its flush from a restored state: the recurrence
    from the values that the cache stands for."""
    lay = make_layer(2, 2, 64, 64, "f32", seed=11)
    lay.S.mul_(0.1)
    cache = StateCache(lay, 1, 8)
    lay.save_state(cache, ints(0), ints(0))
    lay.load_state(cache, ints(1, 0), ints(0, 0))
    torch.cuda.synchronize()
    S = ref.dequantise(codes_of(cache)[0], cache.scale[0].cpu().numpy()).astype(np.float64)
    for w in range(4):
        st = lay.new_step()
        g = torch.Generator(device="cuda").manual_seed(70 + w)
        st.q.copy_(torch.nn.functional.normalize(torch.randn(st.q.shape, generator=g, device="cuda"), dim=-1))
        st.k.copy_(torch.nn.functional.normalize(torch.randn(st.k.shape, generator=g, device="cuda"), dim=-1))
        st.v.normal_(generator=g)
        st.gate.uniform_(0.9, 1.0, generator=g)
        st.beta.uniform_(0, 1, generator=g)
        assert lay.read(st) == 0 and lay.flush(st) == 0
        q, k, v, al, be = [x[1].double().cpu().numpy() for x in (st.q, st.k, st.v, st.gate, st.beta)]
        o = np.zeros((2, 64))
        for h in range(2):
            oo, S[h], _ = ref.delta_rule(q[h][None], k[h][None], v[h][None], al[h][None], be[h][None], S[h])
            o[h] = oo[0]
    got = st.o[1].double().cpu().numpy()
    assert np.linalg.norm(got - o) <= 1e-5 * np.linalg.norm(o)


@pytest.mark.parametrize("bits", [8, 4])
def test_the_last_of_very_many_slots(bits):
    """Codes whose offsets pass 32 bits (2^31 elements of 8 bits, 2^32 of 4)."""
    H, dk, dv = 16, 128, 128
    slots = (1 << (13 if bits == 8 else 14)) + 3
    lay = DecodeLayer("gdn", 2, H, H, dk, dv, 2, "bf16", "bf16", np.arange(H + 1, dtype=np.int32) * 2)
    g = torch.Generator(device="cuda").manual_seed(9)
    lay.S.copy_(torch.randn(lay.S.shape, generator=g, device="cuda"))
    S0, cache = lay.S.clone(), StateCache(lay, slots, bits)
    assert cache.codes.numel() > 1 << 31
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    assert lay.save_state(cache, dev(0, 1), dev(slots - 1, 0)) == 0
    assert lay.load_state(cache, dev(1, 0), dev(slots - 1, 0)) == 0
    # half a step of each block's scale, and the product's rounding
    step = S0.abs().unflatten(-1, (-1, 32)).amax(-1) / (127 if bits == 8 else 7)
    for b in (0, 1):
        err = (lay.S[b] - S0[1 - b]).abs().unflatten(-1, (-1, 32)).amax(-1)
        assert (err <= 0.5001 * step[1 - b]).all()
    assert not cache.codes[1:slots - 1:512].any() and lay.error_word() == 0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_many_sequences_at_once(bits, dk, dv):
    """More tiles than are split over workgroups, values near the borders between
    codes among them."""
    B, H = 131, 5
    lay = make_layer(B, H, dk, dv, "bf16", seed=dk + bits)
    m = 127 if bits == 8 else 7
    blocks = lay.S.unflatten(-1, (-1, 32))
    top = blocks[..., :1].abs() + 1
    g = torch.Generator(device="cuda").manual_seed(17)
    odd = torch.randint(-m, m, blocks.shape, generator=g, device="cuda") + 0.5
    near = (odd / m * top).clamp(-top, top)              # a half, or a rounding beside it
    near = torch.nextafter(near, torch.randn(near.shape, generator=g, device="cuda") * 9)
    blocks.copy_(torch.where(torch.rand(near.shape, generator=g, device="cuda") < 0.3, near, blocks.clamp(-top, top)))
    blocks[..., :1] = top
    cache = StateCache(lay, B, bits)
    order = torch.randperm(B, generator=torch.Generator().manual_seed(3)).int().cuda()
    assert lay.save_state(cache, order, torch.arange(B, dtype=torch.int32, device="cuda")) == 0
    S, seqs = lay.S.cpu().numpy(), order.tolist()
    codes, scales = codes_of(cache), cache.scale.cpu().numpy()
    for slot, b in enumerate(seqs):
        c, s = ref.quantise(S[b], bits)
        assert np.array_equal(codes[slot], c) and np.array_equal(scales[slot], s)
    assert lay.error_word() == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_the_largest_fp32_values_are_read_back_finite(bits):
    """Half a step of the scale, and the scale's own rounding (down, for the
    largest in 8 bits)."""
    lay = make_layer(2, 2, 64, 64)
    top = torch.finfo(torch.float32).max
    lay.S[0, 0] = torch.linspace(-top, top, 64, device="cuda", dtype=torch.float64).clamp(-top, top).float()
    lay.S[0, 1, :, 32:] = -top
    S0 = lay.S[0].double().cpu().numpy()
    cache = StateCache(lay, 1, bits)
    assert lay.save_state(cache, ints(0), ints(0)) == 0
    assert lay.load_state(cache, ints(1), ints(0), prime=False) == 0
    torch.cuda.synchronize()
    m = 127 if bits == 8 else 7
    amax = np.abs(S0.reshape(2, 64, 2, 32)).max(-1, keepdims=True).repeat(32, -1).reshape(S0.shape)
    got = lay.S[1].double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - S0) <= (0.5 / m + 2.0 ** -22) * amax).all()
