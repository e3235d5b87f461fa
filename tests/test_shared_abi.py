"""Groups that share a prefix and 8-bit index keys without a GPU: refusals on
the host, before anything is enqueued."""
import ctypes as C

import pytest
import torch

from test_abi import _problem

FAKE = 1 << 30
GROUPS = dict(num_seqs=3, total_rows=3, max_rows_per_seq=1, num_decode_seqs=3, block_table=FAKE, block_table_stride=64,
              page_size=64, num_groups=2, max_shared_len=1024, max_group_rows=2, group_starts=FAKE, group_shared=FAKE)


def _groups(**over):
    return _problem(**dict(GROUPS, **over))


@pytest.mark.parametrize("over,status", [
    (dict(), 0), (dict(num_groups=3), 0), (dict(max_shared_len=0), 0), (dict(max_shared_len=4096), 0),
    (dict(num_groups=-1), 1), (dict(num_groups=4), 1), (dict(group_starts=None), 1), (dict(group_shared=None), 1),
    (dict(group_starts=FAKE + 2), 1), (dict(group_shared=FAKE + 1), 1), (dict(max_shared_len=-1), 1),
    (dict(max_shared_len=4097), 1), (dict(max_group_rows=0), 1), (dict(max_group_rows=4), 1),
    (dict(block_table=None), 2), (dict(total_rows=30, max_rows_per_seq=9, num_decode_seqs=-1), 2),
    (dict(ik_dtype=2), 1), (dict(ik_dtype=1), 1), (dict(ik_dtype=1, ik_exp=FAKE + 8), 1), (dict(ik_dtype=1, ik_exp=FAKE), 0),
    (dict(kv_dtype=1, k_scale=FAKE, v_scale=FAKE), 0),
])
def test_groups_checked_on_host(over, status):
    import block_sparse_attention_index_gb300 as m
    n = C.c_size_t(0)
    for size in (m.lib().msa_workspace_size, m.lib().msa_dense_workspace_size):
        assert size(C.byref(_groups(**over)), C.byref(n)) == status
        assert (n.value % 256 == 0 and n.value >= 256) if status == 0 else m.lib().msa_last_error()


def test_the_dense_workspace_holds_the_parts():
    """Two parts of max_group_rows x G rows for each item of a group's prefix, two of max_rows_per_seq x G for each of a
    sequence's own positions, 520 bytes a row."""
    import block_sparse_attention_index_gb300 as m
    L, n = m.lib(), C.c_size_t(0)
    assert L.msa_dense_workspace_size(C.byref(_groups()), C.byref(n)) == 0
    rows = 2 * (2 * 4 * 2 * 16) + 3 * 4 * 2 * 16
    assert n.value >= rows * 520
    f, o, ws = C.c_void_p(FAKE), C.c_void_p(2 * FAKE), C.c_void_p(1 << 20)
    p = _groups()
    assert L.msa_dense_forward(C.byref(p), f, f, f, o, ws, n.value - 1, None) == 3
    assert L.msa_dense_forward(C.byref(p), f, f, f, o, None, n.value, None) == 3
    assert L.msa_dense_forward(C.byref(p), f, f, f, o, C.c_void_p((1 << 20) + 16), n.value, None) == 3
    assert L.msa_dense_forward(C.byref(p), f, f, f, f, ws, n.value, None) == 1


def test_problem_checks_its_groups():
    import block_sparse_attention_index_gb300 as m

    def problem(shared, seqs=((1, 300), (2, 400), (1, 90)), **kw):
        return m.Problem(2, 4, seqs, "cpu", block_table=[[0] * 8] * 3, page_size=64, cache_tokens=1024, shared=shared, **kw)

    pb = problem([(2, 256), (1, 64)])
    assert pb.c.num_groups == 2 and pb.c.max_shared_len == 256 and pb.c.max_group_rows == 3
    assert pb.group_starts.tolist() == [0, 2, 3] and pb.group_shared.tolist() == [256, 64]
    assert problem(None).c.num_groups == 0 and problem([]).c.num_groups == 0
    assert problem([(2, 299)]).c.num_groups == 1
    for bad in ([(2, 300)], [(0, 64)], [(4, 64)], [(2, 64), (2, 64)], [(1, -1)], [(2, 256), (1, 90)]):
        with pytest.raises(ValueError):
            problem(bad)
    with pytest.raises(TypeError):
        problem(None, ik_exp=torch.zeros(1024, 2))
    with pytest.raises(ValueError):
        problem(None, ik_exp=torch.zeros(1024, 4, dtype=torch.int8))
    with pytest.raises(ValueError):
        problem(None, ik_exp=torch.zeros(2, 1024, dtype=torch.int8).T)
    assert problem(None, ik_exp=torch.zeros(1024, 2, dtype=torch.int8)).c.ik_dtype == 1
