"""msa_dense_forward with groups over contexts so long that a CTA's share of an
item is more than the 32,768 keys that one sum in tensor memory takes: the
pieces are added up in the workspace."""
import pytest
import torch

from shared_common import SharedBatch
from test_gpu_shared_prefix import behind

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
PREFIX = 12 * 32768


def batch(count, own, **kw):
    """8 heads: 5.4 million keys and more of a head, 35,000 a CTA and more."""
    return SharedBatch(behind(PREFIX, [own + 61 * i for i in range(count)]), [(count, PREFIX)], 8, 16, page=256, seed=count, **kw)


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("count,own", [(4, 70000), (9, 40000)])
def test_shares_of_several_pieces(count, own, int8, out):
    """4 sequences: one M tile, its two stages with parts of their own; 9: two M tiles."""
    batch(count, own, int8=int8, out=out).check()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_long_contexts_behind_a_short_prefix(out):
    SharedBatch([(3, 700000), (1, 99), (8, 650000)], [(3, 64)], 8, 16, page=4096, out=out, seed=2).check()


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("large,at", [(65536 + 10, 65536 - 10), (65536 - 10, 65536 + 10)])
def test_a_value_of_no_weight_in_another_piece(large, at, bad, out):
    """One key scores 256 more than all others; on the other side of a piece's end a value is not finite."""
    a = batch(4, 70000, out=out, scale=1.0)
    a.q.fill_(1.0)
    a.k.zero_()
    a.k[a.rows_of(0, torch.tensor([large], device="cuda"))] = 2.0
    a.v[a.rows_of(0, torch.tensor([at], device="cuda")), :, 3] = bad
    got = a.run()
    assert not torch.isfinite(got[..., 3]).any()
    got[..., 3] = 0
    want = a.v[a.rows_of(0, torch.tensor([large], device="cuda"))][0].repeat_interleave(16, 0)[None].expand_as(got).clone()
    want[..., 3] = 0
    assert torch.equal(got, want.to(out))


@pytest.mark.parametrize("out", [BF16, FP32])
def test_pieces_without_a_score(out):
    """Keys of minus infinity for the rows of one piece, or of all but one: they have no weight."""
    a = batch(4, 70000, out=out)
    a.q.abs_()
    t = torch.arange(PREFIX, device="cuda")
    rows = a.rows_of(0, t)
    for hidden in (t < 32768, t >= 32768):
        a.k.copy_(torch.randn(a.k.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16())
        a.k[rows[hidden]] = -float("inf")
        got = a.run().double()
        # the formula over the others
        b, h, first = 1, 5, 1
        seen = torch.cat([rows[~hidden], a.rows_of(b, torch.arange(PREFIX, a.seqs[b][1], device="cuda"))])
        k, v, q = a.k[seen, h].double(), a.v[seen, h].double(), a.q[first, h * 16:h * 16 + 16].double()
        w = torch.softmax(a.scale * q @ k.T, 1)
        bits = 2.0 ** -8 if out == BF16 else 2.0 ** -24
        A = a.scale * (q.abs() @ k.abs().T).amax(1)
        rel = 2 * 133 * 2.0 ** -24 * A + 2.0 ** -22 + 2 * len(seen) * 2.0 ** -24 + bits
        bound = (w @ v.abs()) * rel[:, None] + (w @ v).abs() * torch.finfo(out).eps / 2
        assert ((got[first, h * 16:h * 16 + 16] - w @ v).abs() <= bound).all()
