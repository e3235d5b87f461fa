"""Values that are not finite in what a group's rows see: they show in the
outputs, however small their weights are."""
import pytest
import torch

from shared_common import SharedBatch
from test_gpu_shared_prefix import behind

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("large,at", [("own", 5), ("own", 700), ("prefix", 1100), ("window", 5), ("window", 1100), ("prefix", 1221)])
def test_a_value_of_no_weight(large, at, bad, out):
    """One key scores 256 more than all others, whose weights are then 0 in 32 bits; one value of another part of the keys is
    not finite (the prefix ends at 1,024, the own positions at 1,220, the window has two)."""
    a = SharedBatch(behind(1024, [196, 196], 2), [(2, 1024)], 2, 16, out=out, scale=1.0)
    a.q.fill_(1.0)
    a.k.zero_()
    t = {"prefix": 300, "own": 1200, "window": 1220}[large]
    for b in range(2):
        a.k[a.rows_of(b, torch.tensor([t], device="cuda"))] = 2.0
        a.v[a.rows_of(b, torch.tensor([at], device="cuda")), 1, 3] = bad
    got = a.run().view(4, 2, 16, 128)
    sees = torch.ones(4, dtype=torch.bool) if at < 1221 else torch.tensor([False, True, False, True])
    assert not torch.isfinite(got[sees.cuda(), 1, :, 3]).any()
    got[sees.cuda(), 1, :, 3] = 0
    assert torch.isfinite(got).all()
    v = torch.stack([a.v[a.rows_of(b, torch.tensor([t], device="cuda"))][0] for b in (0, 0, 1, 1)])[:, :, None].expand_as(got).clone()
    v[sees.cuda(), 1, :, 3] = 0
    assert torch.equal(got, v.to(out))  # one weight of 1: its value exactly
