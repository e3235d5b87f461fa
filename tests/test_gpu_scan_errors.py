"""What any CTA of an index scan finds wrong reaches the error word of the call,
whichever sequences the batch begins with, and nothing of an earlier call does."""
import pytest
import torch

from gpu_common import msa
from test_gpu_index8 import Sparse

pytestmark = pytest.mark.gpu


def word(a, codes, ws=None, **kw):
    m = msa()
    pb = m.Problem(a.H, a.G, a.seqs, "cuda", **dict(a.kw, ik_exp=a.exp if codes else None, **kw))
    if ws is None:
        ws = pb.workspace()
        ws.fill_(0xFF)
    m.forward(pb, a.q, a.iq, a.k, a.v, a.codes if codes else a.values(), workspace=ws)
    torch.cuda.synchronize()
    return m.error_word(ws)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("first", [[], [(40, 700)], [(8, 300)], [(300, 300), (1, 2)]])
def test_a_bad_page_anywhere(first, codes):
    """The page of one block in turn, of a sequence of 300 blocks (two to a CTA): a few of them are read again by the
    attention, the others by one CTA of the scan alone.  The batch begins with prompt chunks or drafted windows, so that the
    first CTA of the attention has a row of its own or none."""
    a = Sparse(first + [(1, 300 * 64)], 2, 4, 64)
    table, b = a.kw["block_table"], len(first)
    for counted in ("auto", 0):
        assert word(a, codes, num_decode_rows=counted) == 0
        for page in range(0, 300, 23):
            keep = int(table[b, page])
            table[b, page] = 1 << 20
            assert word(a, codes, num_decode_rows=counted) == msa().ERR_BAD_METADATA, (counted, page)
            table[b, page] = keep


def test_the_word_is_of_the_last_call():
    a = Sparse([(1, 20000), (3, 5000)], 4, 4, 64)
    pb = msa().Problem(a.H, a.G, a.seqs, "cuda", **a.kw)
    ws = pb.workspace()
    assert word(a, False, ws) == 0
    keep = a.kw["block_table"].clone()
    a.kw["block_table"][0, 170] = -1
    assert word(a, False, ws) == msa().ERR_BAD_METADATA
    a.kw["block_table"].copy_(keep)
    assert word(a, False, ws) == 0 and word(a, True, ws) == 0


def test_no_row_of_the_decode_kernels():
    """The host does not know the families and every sequence is a prompt chunk: the scan has nothing to do."""
    a = Sparse([(40, 700), (9, 3000)], 2, 4, 64)
    for codes in (False, True):
        assert word(a, codes, num_decode_seqs=-1, num_decode_rows=0) == 0
