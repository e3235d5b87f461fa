"""msa_dense_forward where a bounded wait has given up, and where a call's
own work takes longer than a wait may."""
import pytest
import torch

from gpu_common import msa
from test_gpu_dense import Batch

pytestmark = pytest.mark.gpu


def test_split_items_are_not_joined_after_a_wait_gave_up():
    """What the join reads may then never have been written.  The bit comes from the diagnostic entry point, on another
    stream, 5 ms into a call that takes some 70 (its last part computes rows again for the NaN); 40 rows are too few
    items for every SM, so that both kernels run."""
    m = msa()
    L = 1 << 21
    b = Batch([(40, L)], 1, 16, False, 0, torch.bfloat16)
    b.v[b.starts[0] + L - 1] = float("nan")
    ws, out = b.dirty_workspace(), torch.full_like(b.pb.new_out(), 7.0)
    other = torch.cuda.Stream()
    # (kernels are loaded by their first launch, which may wait for the GPU)
    m.check_wait_timeout(torch.zeros(256, dtype=torch.uint8, device="cuda"), 1)
    m.dense_forward(b.pb, b.q, b.k, b.v, workspace=ws)
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    m.dense_forward(b.pb, b.q, b.k, b.v, out=out, workspace=ws)
    end.record()
    with torch.cuda.stream(other):
        m.check_wait_timeout(ws, 5000)
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 10  # (else the bit came too late to tell)
    assert m.error_word(ws) == m.ERR_WAIT_TIMEOUT
    assert (out == 7).all()
    m.dense_forward(b.pb, b.q, b.k, b.v, out=out, workspace=ws)  # the next call is as any other
    torch.cuda.synchronize()
    assert m.error_word(ws) == 0
    assert torch.isfinite(out[:39]).all() and torch.isnan(out[39]).all() and not (out == 7).all(-1).any()


def test_work_that_outlasts_a_wait_is_waited_for():
    """Rows that are computed again over 2^21 positions take a CTA 2.5 s or more, while its other warps wait for their
    next item."""
    m = msa()
    L, n = 1 << 21, 640
    b = Batch([(n, L)], 8, 16, False, 0, torch.bfloat16, seed=2)
    at = b.starts[0]
    b.v[at + L - 1] = float("nan")  # the last row sees it; the 15 rows of its tiles before it are computed again
    got = b.run()
    assert torch.isnan(got[n - 1]).all()
    assert torch.isfinite(got[:n - 1]).all()
    # weights to 2^-8 each, half a step of bf16, the sums' 2 L 2^-24 as in 64 bits' bound (of |values| of the same size)
    for row, head in ((n - 2, 0), (n - 16, 77), (n - 17, 127), (0, 5), (n // 2, 40)):
        h, end = head // 16, at + L - n + row + 1
        x = (b.k[at:end, h].double() @ b.q[row, head].double()) * b.scale
        w = torch.softmax(x, 0)
        v = b.v[at:end, h].double()
        ref, bound = w @ v, (w @ v.abs()) * (2.0 ** -8 + 2.0 ** -12) + 2.0 ** -8 * (w @ v).abs()
        assert ((got[row, head].double() - ref).abs() <= bound).all()
