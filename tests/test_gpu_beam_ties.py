"""Equal beams are ties: rows of the same logits and scores have the same candidates,
wherever in memory the rows begin, so that the lowest b * vocab + j comes first."""
import pytest
import torch

from tests import test_gpu_beams as beams

pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from ssm_decode_amd.layer import TORCH_DTYPE
    from ssm_decode_amd.serving import BeamSearch


def equal_rows(n, k, V, pad, skip, act, seed):
    """A random row a group, the group's rows V + pad elements apart, from element `skip` of their memory."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    row = (2 * torch.randn((n, 1, V), generator=g, device="cuda")).to(TORCH_DTYPE[act])
    x = torch.empty(skip + n * k * (V + pad), device="cuda", dtype=row.dtype)[skip:].view(n * k, V + pad)[:, :V]
    x.copy_(row.expand(n, k, V).reshape(n * k, V))
    return x


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,V,pad,skip", [(2, 2, 97, 0, 0), (1, 4, 8192, 1, 0), (3, 5, 50001, 0, 0), (2, 8, 50257, 0, 3), (2, 16, 30011, 2, 1),
                                            (1, 16, 128001, 0, 0), (4, 4, 128000, 0, 0), (1, 9, 20000, 3, 5)])
def test_equal_beams_go_to_the_lowest(n, k, V, pad, skip, act):
    for seed in range(4):
        x = equal_rows(n, k, V, pad, skip, act, seed)
        s = torch.full((n, k), -1.25, device="cuda")
        search = BeamSearch(n, k, V)
        none = torch.zeros_like(search.ended)
        assert search.select(x, s, none) == 0
        beams.check(search, x, s, none)
        scores = search.scores.view(torch.int32)
        tops = search.tokens == search.tokens[:, :1]
        assert (scores[tops] == scores[:, :1].expand_as(scores)[tops]).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_row_counts_alike_wherever_it_begins(act):
    """One beam at every place of 16 bytes: the score of the same row, to the bit."""
    V, seen = 50001, set()
    for skip in range(8):
        x = equal_rows(1, 1, V, 0, skip, act, 7)
        search = BeamSearch(1, 1, V)
        assert search.select(x) == 0
        seen.add((int(search.tokens[0, 0]), int(search.scores.view(torch.int32)[0, 0])))
    assert len(seen) == 1
