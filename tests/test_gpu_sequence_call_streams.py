"""Temporaries dropped behind a convolution, a selection or a reordering on a stream
that is given, which is kept busy meanwhile."""
import pytest
import torch

from tests import test_gpu_beams as beams
from tests import test_gpu_conv as conv
from tests.test_gpu_sequence_streams import busy
from tests.test_gpu_serving_streams import reused

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.serving import BeamSearch


def place(*tensors):
    return {t.data_ptr() for t in tensors}, [t.numel() * t.element_size() for t in tensors]


def test_a_convolutions_lists_and_rows_dropped():
    c = conv.Case(300, 3, seed=710)
    at, seqs, has = [0, 200, 201, 300], [2, 0, 1], [1, 0, 1]
    lists = [conv.ints(at), conv.ints(seqs), conv.ints(has)]
    x = c.x.contiguous()
    where = place(*lists, x)
    side = busy()
    keep, c.x = c.x, x
    assert c.call(seq_start=lists[0], seqs=lists[1], has_state=lists[2], stream=side.cuda_stream) == 0
    c.x = keep
    del x, lists
    assert not side.query()
    assert not reused(*where)
    assert not side.query()
    torch.cuda.synchronize()
    c.check(at, seqs, has)


def test_a_selections_logits_dropped():
    n, k, V = 3, 4, 20011
    x, s = beams.inputs(n, k, V, "bf16", seed=711)
    search = BeamSearch(n, k, V)
    e = torch.zeros_like(search.ended)
    given = [x.clone(), s.clone(), e.clone()]
    where = place(*given)
    side = busy()
    assert search.select(*given, stream=side.cuda_stream) == 0
    del given
    assert not side.query()
    assert not reused(*where)
    assert not side.query()
    torch.cuda.synchronize()
    beams.check(search, x, s, e)


def test_a_reorderings_parents_dropped():
    lay, cv, held = beams.make("mamba2", 24, H=8, G=4, dk=64, dv=64, W=4, act="bf16", seed=712)
    at = torch.tensor([b // 3 * 3 + (2 * b + b // 3) % 3 for b in range(24)], dtype=torch.int32, device="cuda")
    want = {n: x[at.long()].clone() for n, x in held.items()}
    where = place(at)
    side = busy()
    assert lay.reorder(at, 3, convs=(cv,), stream=side.cuda_stream) == 0
    del at
    assert not side.query()
    assert not reused(*where)
    assert not side.query()
    torch.cuda.synchronize()
    for n, x in held.items():
        assert torch.equal(x, want[n]), n
