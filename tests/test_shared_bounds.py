"""The workspaces of batches with groups hold what device metadata can make the
kernels write, whatever it says: sizes on the host, no GPU."""
import ctypes as C

import pytest

from test_shared_abi import _groups


@pytest.mark.parametrize("seqs,rows,most,length,heads", [
    (2, 64, 1, 65536, 4), (2, 6, 1, 640, 4), (3, 3, 1, 4096, 1), (16, 128, 8, 4096, 8), (5, 9, 2, 100000, 2)])
def test_a_slot_for_every_row(seqs, rows, most, length, heads):
    """With groups the pooled scores (4 bytes a head and block) lie by query row: the workspace has to hold those of
    total_rows rows, also where that is more than num_seqs x max_rows_per_seq (rows behind the last sequence)."""
    import block_sparse_attention_index_gb300 as m
    p = _groups(num_seqs=seqs, total_rows=rows, max_rows_per_seq=most, num_decode_seqs=seqs, max_cache_len=length,
                num_kv_heads=heads, max_group_rows=rows, max_shared_len=length, block_table_stride=-(-length // 64),
                cache_tokens=1 << 20)
    n = C.c_size_t(0)
    assert m.lib().msa_workspace_size(C.byref(p), C.byref(n)) == 0
    blocks = -(-length // 64)
    assert n.value >= rows * heads * (4 * blocks + 16 * 4 + 4)  # and the kept blocks
