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


@pytest.mark.parametrize("seqs,rows,heads,most_mb", [(64, 1, 4, 40), (64, 8, 4, 100), (256, 8, 4, 256), (4096, 8, 8, 6800)])
def test_the_dense_workspace_does_not_grow_with_the_lengths(seqs, rows, heads, most_mb):
    """Parts are as many as items and CTAs: two of rows x 16 pairs for each (sequence, head), two of 128 for each 256 pairs
    of a group and head, and for each of up to 160 CTAs (520 bytes a pair)."""
    import block_sparse_attention_index_gb300 as m
    sizes = []
    for length in (4096, 1 << 17, 1 << 21):
        p = _groups(num_seqs=seqs, total_rows=seqs * rows, max_rows_per_seq=rows, num_decode_seqs=seqs, max_cache_len=length,
                    num_kv_heads=heads, group_size=16, max_group_rows=seqs * rows, max_shared_len=length, num_groups=2,
                    block_table_stride=length // 64, cache_tokens=1 << 24)
        n = C.c_size_t(0)
        assert m.lib().msa_dense_workspace_size(C.byref(p), C.byref(n)) == 0
        sizes.append(n.value)
    assert sizes[0] == sizes[1] == sizes[2] <= most_mb << 20
