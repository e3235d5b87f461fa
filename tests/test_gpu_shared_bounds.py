"""Device metadata that breaks the host's bounds, in batches with groups: it is
reported, and nothing outside the workspace is written."""
import pytest
import torch

from gpu_common import msa
from test_gpu_shared_sparse import Batch, behind

pytestmark = pytest.mark.gpu


def guarded(pb, size):
    """A workspace with 4 MB behind it that nobody may write."""
    store = torch.full((size + (4 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    return store[:size], store[size:]


def forward(a, pb):
    """(error word, guard untouched, out)"""
    m = msa()
    ws, guard = guarded(pb, pb.workspace_size())
    out = torch.full_like(pb.new_out(), float("nan"))
    m.forward(pb, a.q, a.iq, a.k, a.v, a.ik, out=out, workspace=ws)
    torch.cuda.synchronize()
    return m.error_word(ws), bool((guard == 0xA5).all()), out


@pytest.mark.parametrize("index8", [False, True])
@pytest.mark.parametrize("starts", [[0, 1, 64], [0, 3, 6], [0, 33, 34], [0, 1, 9], [0, 63, 64]])
def test_more_rows_than_the_host_says(starts, index8):
    """Two sequences of one row each for the host, rows behind them; the device gives them more."""
    a = Batch(behind(4096, [100, 300]), [(2, 4096)], 4, 8, index8=index8, spare_rows=62)
    pb = a.problem(True)
    pb.c.max_group_rows = 64
    pb.cu_rows.copy_(torch.tensor(starts, dtype=torch.int32))
    word, intact, _ = forward(a, pb)
    assert intact and word == msa().ERR_BAD_METADATA


@pytest.mark.parametrize("first", [5, 50, 62])
def test_rows_that_begin_later(first):
    """Rows before the first sequence: its scores lie at its rows' slots all the same."""
    a = Batch(behind(4096, [100, 300]), [(2, 4096)], 4, 8, spare_rows=62)
    pb = a.problem(True)
    pb.cu_rows.copy_(torch.tensor([first, first + 1, first + 2], dtype=torch.int32))
    word, intact, out = forward(a, pb)
    assert intact and word == 0
    b = a.problem(False)
    b.cu_rows.copy_(pb.cu_rows)
    assert torch.equal(out[first:first + 2], forward(a, b)[2][first:first + 2])
    assert torch.isnan(out[:first]).all() and torch.isnan(out[first + 2:]).all()


def test_rows_past_the_total():
    a = Batch(behind(1280, [100, 300], 2), [(2, 1280)], 2, 8)
    pb = a.problem(True)
    pb.cu_rows.copy_(torch.tensor([1, 3, 5], dtype=torch.int32))
    word, intact, _ = forward(a, pb)
    assert intact and word == msa().ERR_BAD_METADATA


@pytest.mark.parametrize("starts", [[0, 3, 0, 3], [0, 3, 2, 3], [3, 0, 0, 3], [1, 0, 3, 1], [0, 3, -1, 3], [0, 4, 0, 3],
                                    [0, 2 ** 31 - 1, 0, 3]])
@pytest.mark.parametrize("index8", [False, True])
def test_groups_that_do_not_ascend(starts, index8):
    """Three groups whose starts go down again: some of them overlap."""
    a = Batch(behind(1280, [100, 300, 5], 2), [(1, 1280), (1, 1280), (1, 1280)], 2, 8, index8=index8)
    pb = a.problem(True)
    pb.c.max_group_rows = 6
    pb.group_starts.copy_(torch.tensor(starts, dtype=torch.int32))
    word, intact, _ = forward(a, pb)
    assert intact and word == msa().ERR_BAD_METADATA
    ws, guard = guarded(pb, pb.dense_workspace_size())
    msa().dense_forward(pb, a.q, a.k, a.v, workspace=ws)
    torch.cuda.synchronize()
    assert bool((guard == 0xA5).all()) and msa().error_word(ws) == msa().ERR_BAD_METADATA


def test_more_parts_than_the_host_allows_for():
    """64 groups that overlap, each of 64 rows and two parts: the workspace has room for those of 64 rows in all."""
    seqs = behind(33000, [i for i in range(64)])
    a = Batch(seqs, [(1, 33000)] * 64, 1, 16)
    pb = a.problem(True)
    pb.c.max_group_rows = 64
    ws, guard = guarded(pb, pb.dense_workspace_size())
    good = msa().dense_forward(pb, a.q, a.k, a.v, workspace=ws).clone()
    torch.cuda.synchronize()
    assert msa().error_word(ws) == 0 and bool((guard == 0xA5).all()) and torch.isfinite(good).all()
    pb.group_starts.copy_(torch.tensor([64 * (i % 2) for i in range(65)], dtype=torch.int32))
    msa().dense_forward(pb, a.q, a.k, a.v, workspace=ws)
    torch.cuda.synchronize()
    assert msa().error_word(ws) == msa().ERR_BAD_METADATA and bool((guard == 0xA5).all())
    word, intact, _ = forward(a, pb)
    assert intact and word == msa().ERR_BAD_METADATA


def test_a_line_longer_than_any_batch():
    """256 groups that overlap, each of 4,096 rows and 2^15 blocks: 2^31 and more units of time in all."""
    m = msa()
    B, n, most = 512, 8, 1 << 21
    table = torch.zeros(B, most // 64, dtype=torch.int32, device="cuda")
    pb = m.Problem(1, 1, [(n, 264)] * B, "cuda", block_table=table, page_size=64, cache_tokens=64, shared=[(1, 256)] * B)
    pb.c.max_cache_len = pb.c.max_shared_len = most
    pb.c.max_group_rows = B * n
    pb.group_starts.copy_(torch.tensor([B * (i % 2) for i in range(B + 1)], dtype=torch.int32))
    pb.group_shared.fill_(most)
    q = torch.zeros(B * n, 1, 128, dtype=torch.bfloat16, device="cuda")
    iq = torch.zeros(B * n, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(64, 1, 128, dtype=torch.bfloat16, device="cuda")
    ik = torch.zeros(64, 1, 64, dtype=torch.bfloat16, device="cuda")
    ws, guard = guarded(pb, pb.workspace_size())
    m.forward(pb, q, iq, k, k, ik, workspace=ws)
    torch.cuda.synchronize()
    assert m.error_word(ws) == m.ERR_BAD_METADATA and bool((guard == 0xA5).all())
