"""Prompts and caches dropped while calls on another stream still use them."""
import pytest
import torch

from tests.prompt_bounds import rule, state_off, wrong_outputs
from tests.test_gpu_prefill import make_layer, make_tokens

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.serving import Prompts, StateCache

BUSY = 1 << 27          # cycles that the other stream is kept from the call


def reused(addresses, sizes):
    """Whether new tensors of these sizes come to lie at one of the addresses."""
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    return bool(addresses & {t.data_ptr() for t in new})


@pytest.mark.parametrize("given", ["handle", "current"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_prompts_dropped_behind_their_call(act, given):
    lens = [300, 150]
    lay = make_layer(2, 3, 128, 128, act, seed=400)
    tok = make_tokens(450, 3, 128, 128, act, seed=401)
    S0 = lay.S.clone()
    pr = Prompts(lay, *tok, torch.tensor([0, 300, 450], dtype=torch.int32, device="cuda"))
    at, size = {pr.work.data_ptr(), pr.seq_start.data_ptr()}, [pr.work.numel(), 12]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    if given == "handle":
        assert lay.prefill(pr, stream=side.cuda_stream) == 0
    else:
        with torch.cuda.stream(side):
            assert lay.prefill(pr) == 0
    del pr
    assert not side.query()
    assert not reused(at, size)
    assert not side.query()
    torch.cuda.synchronize()
    for i, (a, n) in enumerate(((0, 300), (300, 150))):
        o, S, scale = rule(*(x[a:a + n] for x in tok[:5]), S0[i])
        assert wrong_outputs(tok[5][a:a + n], o, scale, 128) == (0, 0)
        assert state_off(lay.S[i], S, 128) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_a_cache_dropped_behind_its_call(bits):
    lay = make_layer(4, 2, 64, 64, "bf16", seed=402)
    idx = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1], [1, 0], [2, 3])]
    cache = StateCache(lay, 2, bits)
    assert lay.save_state(cache, idx[0], idx[1]) == 0
    assert lay.load_state(cache, idx[2], idx[1]) == 0
    want = lay.S[2:].clone()
    lay.S[2:] = 0
    at, size = {cache.codes.data_ptr(), cache.scale.data_ptr()}, [cache.codes.numel(), 4 * cache.scale.numel()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    assert lay.load_state(cache, idx[2], idx[1], stream=side.cuda_stream) == 0
    del cache
    assert not reused(at, size)
    assert not side.query()
    torch.cuda.synchronize()
    assert torch.equal(lay.S[2:], want)


def test_prompts_of_another_stream_on_the_default_one():
    """Made on a stream of its own, called on the default stream (handle 0)."""
    lay = make_layer(1, 2, 64, 64, "bf16", seed=403)
    tok = make_tokens(200, 2, 64, 64, "bf16", seed=404)
    S0 = lay.S.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pr = Prompts(lay, *tok, torch.tensor([0, 200], dtype=torch.int32, device="cuda"))
        at, size = {pr.work.data_ptr()}, [pr.work.numel()]
    side.synchronize()
    torch.cuda._sleep(BUSY)
    assert lay.prefill(pr) == 0
    del pr
    with torch.cuda.stream(side):
        assert not reused(at, size)
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    o, S, scale = rule(*tok[:5], S0[0])
    assert wrong_outputs(tok[5], o, scale, 64) == (0, 0) and state_off(lay.S[0], S, 64) == 0
