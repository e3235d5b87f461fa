"""msa_dense_forward on caches whose scales, keys or lengths strain its number
formats."""
import pytest
import torch

from gpu_common import msa
from test_gpu_dense import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("first", [32, 70, 128])
def test_scores_of_minus_infinity_weigh_nothing(first, out, n):
    """Keys with an infinity against a negative query, from the first position on; a chunk's last value is NaN, so
    that rows before it are computed again.  The other weights sum to 1 and are off by 2^-8 of themselves at most, the
    output by half a step of bf16, 2^-8 of itself: with the fp32 sums (below 2^-10) less than 2.5 2^-8 max |v|."""
    b = Batch([(n, 300)], 2, 16, False, 0, out, seed=first)
    rows = b.rows_of(0, torch.arange(300, device="cuda"))
    b.q[..., 5] = -1 - b.q[..., 5].abs()
    b.k[rows[:first], :, 5] = float("inf")
    ref, _ = b.ref()
    most = b.v[rows].abs().max().double()
    live = n
    if n > 8:
        b.v[rows[-1]] = float("nan")
        live = n - 1
    got = b.run()
    assert ((got.double() - ref).abs() <= 2.5 * 2.0 ** -8 * most)[:live].all()
