"""msa_forward with groups in the forms that servers combine: int8 keys and
values, index keys in bf16 or codes, one index key for all heads, drafted
windows, two calls at once."""
import pytest
import torch

from gpu_common import msa
from test_gpu_shared_sparse import Batch, behind

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G", [(1, 16), (4, 16), (8, 5)])
@pytest.mark.parametrize("index8", [False, True])
@pytest.mark.parametrize("ik_heads", [0, 1])
@pytest.mark.parametrize("rows", [1, 3, 8])
def test_int8_keys_and_values(H, G, rows, ik_heads, index8):
    seqs = behind(1920, [0, 1, 63, 700], rows) + behind(320, [5, 2000], rows) + [(1, 1), (rows, 1500)]
    Batch(seqs, [(4, 1920), (2, 320)], H, G, index8=index8, ik_heads=ik_heads, kv_int8=True, seed=rows).check()


@pytest.mark.parametrize("page", [128, 1024])
@pytest.mark.parametrize("kv_int8", [False, True])
def test_pages(page, kv_int8):
    Batch(behind(2048, [1, 1500, 30], 2) + [(4, 900)], [(3, 2048)], 2, 8, page=page, index8=True, kv_int8=kv_int8, seed=page).check()


def test_two_streams_at_once():
    m = msa()
    a = Batch(behind(8192, [50, 300, 7]), [(3, 8192)], 4, 16, index8=True, seed=1)
    b = Batch(behind(4096, [500, 30], 4) + [(8, 3000)], [(2, 4096)], 4, 16, seed=2)
    want = a.run(), b.run()
    pbs = a.problem(True), b.problem(True)
    made = [(pb.workspace(), pb.new_out(), *pb.new_sel()) for pb in pbs]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        for x, pb, (ws, out, sel, nsel), s in zip((a, b), pbs, made, streams):
            with torch.cuda.stream(s):
                m.forward(pb, x.q, x.iq, x.k, x.v, x.ik, out=out, sel=sel, nsel=nsel, workspace=ws)
    torch.cuda.synchronize()
    for w, (ws, out, sel, nsel) in zip(want, made):
        assert m.error_word(ws) == 0
        assert torch.equal(out, w[0]) and torch.equal(sel, w[1]) and torch.equal(nsel, w[2])


def test_two_calls_of_one_workspace_in_order():
    """A sparse call and a dense one of other batches over the same workspace and stream, several times."""
    m = msa()
    a = Batch(behind(2048, [50, 300, 7], 2), [(3, 2048)], 2, 16, index8=True, seed=3)
    b = Batch(behind(640, [i * 11 for i in range(20)]), [(20, 640)], 2, 16, seed=4)
    pa, pb = a.problem(True), b.problem(True)
    sizes = [p.workspace_size() for p in (pa, pb)] + [p.dense_workspace_size() for p in (pa, pb)]
    ws = torch.full((max(sizes),), 0xFF, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(4):
        got = [m.forward(pa, a.q, a.iq, a.k, a.v, a.ik, workspace=ws), m.dense_forward(pb, b.q, b.k, b.v, workspace=ws),
               m.forward(pb, b.q, b.iq, b.k, b.v, b.ik, workspace=ws), m.dense_forward(pa, a.q, a.k, a.v, workspace=ws)]
        flat = [x for g in got for x in (g if isinstance(g, tuple) else (g,))]
        torch.cuda.synchronize()
        assert m.error_word(ws) == 0
        assert first is None or all(torch.equal(x, y) for x, y in zip(flat, first))
        first = flat
    assert torch.equal(first[0], a.run(False)[0]) and torch.equal(first[4], b.run(False)[0])
