"""msa_dense_forward with host counts that are bounds: a captured step keeps
its counts while the rows of each sequence change on the device."""
import pytest
import torch

from gpu_common import msa
from test_gpu_dense import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("count", [0, 13, 14, 16])
def test_windows_shorter_than_the_host_counts(count, G, int8, out):
    """Up to four drafted rows each, 13 in all: the count unknown, exact, above, and that of full windows."""
    b = Batch([(4, 100), (1, 300), (4, 70), (4, 4)], 2, G, int8, 64, out, spare_rows=3)
    b.pb.c.num_decode_rows = count
    rest = torch.full_like(b.pb.new_out(), 7.0)
    b.check(b.run(out=rest))
    assert (rest[13:] == 7).all()


@pytest.mark.parametrize("count", [0, 64, 65, 512])
@pytest.mark.parametrize("int8", [False, True])
def test_prompts_beside_an_over_count_of_decode_rows(count, int8):
    seqs = [(1, 20 + 90 * i) for i in range(64)] + [(512, 600)]
    b = Batch(seqs, 1, 16, int8, 64, torch.bfloat16)
    b.pb.c.num_decode_rows = count
    b.check()


def test_a_captured_step_follows_its_rows():
    """One graph, captured for full windows, replayed for shorter ones."""
    m = msa()
    full = Batch([(4, 900), (4, 300), (4, 70)], 2, 16)
    ws, out = full.dirty_workspace(), full.pb.new_out()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.dense_forward(full.pb, full.q, full.k, full.v, out=out, workspace=ws)
    for rows in ([4, 4, 4], [1, 4, 2], [2, 1, 1], [1, 1, 1], [3, 1, 4]):
        full.seqs = [(n, L) for n, (_, L) in zip(rows, full.seqs)]
        cu = [0, rows[0], rows[0] + rows[1], sum(rows)]
        full.pb.cu_rows.copy_(torch.tensor(cu, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert m.error_word(ws) == 0
        full.check(out)
        assert (out[sum(rows):] == 7).all()
