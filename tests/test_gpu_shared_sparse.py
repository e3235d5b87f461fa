"""msa_forward with groups of sequences that share a prefix: the index keys of
the prefix are scanned once for the group.  Index queries and keys are small
integers, so that the scores are exact in any order: the same blocks have to be
chosen, and the same outputs given, as by the same call without groups."""
import pytest
import torch

from gpu_common import msa
from shared_common import shared_tables

pytestmark = pytest.mark.gpu


class Batch:
    def __init__(self, seqs, groups, H, G, page=64, index8=False, ik_heads=0, kv_int8=False, claim=None, seed=0, spare_rows=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.seqs, self.groups, self.H, self.G = seqs, groups, H, G
        table, pages = shared_tables(seqs, groups, page, seed)
        T, KH, R = pages * page, 1 if ik_heads == 1 else H, sum(n for n, _ in seqs) + spare_rows
        ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda")  # noqa: E731
        self.R = R
        self.q = torch.randn(R, H * G, 128, generator=g, device="cuda").bfloat16()
        self.iq = ints(-8, 9, R, H, 64).bfloat16()
        self.kw = dict(block_table=table.cuda(), page_size=page, cache_tokens=T, ik_heads=ik_heads, out_dtype=torch.float32,
                       num_decode_seqs=len(seqs))
        self.ik = ints(-127, 128, T, KH, 64).to(torch.int8) if index8 else ints(-8, 9, T, KH, 64).bfloat16()
        if index8:
            self.kw["ik_exp"] = ints(-5, 2, T, KH).to(torch.int8)
        if kv_int8:
            self.k, self.v = (ints(-127, 128, T, H, 128).to(torch.int8) for _ in range(2))
            self.kw.update(k_scale=0.01 + torch.rand(T, H, generator=g, device="cuda") / 64,
                           v_scale=0.01 + torch.rand(T, H, generator=g, device="cuda") / 64)
        else:
            self.k, self.v = (torch.randn(T, H, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
        self.claim = groups if claim is None else claim

    def problem(self, groups):
        pb = msa().Problem(self.H, self.G, self.seqs, "cuda", shared=self.claim if groups else None, **self.kw)
        pb.total_rows = pb.c.total_rows = self.R
        return pb

    def run(self, groups=True, pb=None, error=0):
        m = msa()
        pb = self.problem(groups) if pb is None else pb
        ws = pb.workspace()
        ws.fill_(0xFF)
        out = torch.full_like(pb.new_out(), float("nan"))
        sel, nsel = pb.new_sel()
        sel.fill_(-7), nsel.fill_(-7)
        m.forward(pb, self.q, self.iq, self.k, self.v, self.ik, out=out, sel=sel, nsel=nsel, workspace=ws)
        torch.cuda.synchronize()
        assert m.error_word(ws) == error
        return out, sel, nsel

    def check(self):
        got, want = self.run(True), self.run(False)
        n = sum(c for c, _ in self.seqs)
        assert torch.isfinite(want[0][:n]).all()
        for x, y in zip(got, want):
            assert torch.equal(x[:n], y[:n])
        assert torch.isnan(got[0][n:]).all() and (got[1][n:] == -7).all()


def behind(prefix, own, rows=1):
    return [(rows, prefix + x + rows) for x in own]


@pytest.mark.parametrize("H,G", [(1, 16), (2, 5), (4, 16), (8, 4)])
@pytest.mark.parametrize("index8", [False, True])
@pytest.mark.parametrize("ik_heads", [0, 1])
def test_groups(H, G, index8, ik_heads):
    seqs = behind(2048, [0, 1, 63, 64, 900]) + behind(640, [5, 300, 2000], 3) + [(1, 1), (2, 3000)]
    Batch(seqs, [(5, 2048), (3, 640)], H, G, index8=index8, ik_heads=ik_heads, seed=H).check()


@pytest.mark.parametrize("rows", [1, 2, 5, 8])
@pytest.mark.parametrize("index8", [False, True])
def test_windows(rows, index8):
    Batch(behind(1984, [0, 3, 64, 150, 700], rows), [(5, 1984)], 4, 8, index8=index8, seed=rows).check()


@pytest.mark.parametrize("count", [1, 2, 7, 8, 9, 64, 300])
def test_rows_of_a_group(count):
    Batch(behind(1280, [(37 * i) % 150 for i in range(count)]), [(count, 1280)], 2, 16, seed=count).check()


@pytest.mark.parametrize("claim", [0, 1, 64, 100, 1000, 1300])
def test_shared_positions_of_any_number(claim):
    Batch(behind(1300, [0, 40, 90], 2), [(3, 1300)], 2, 8, page=64, claim=[(3, claim)]).check()


def test_one_group_after_another():
    groups = [(3, 64 * (1 + i % 30)) for i in range(120)]
    seqs = [s for count, p in groups for s in behind(p, [(p * 7 + j * 31) % 90 for j in range(count)])]
    Batch(seqs + [(1, 1 + (i * 13) % 2000) for i in range(50)], groups, 2, 4).check()


def test_sequences_without_rows():
    Batch([(1, 1500), (0, 1400), (8, 1464), (3, 1461), (0, 400), (5, 900), (0, 64), (4, 77)], [(4, 1280)], 2, 16, spare_rows=6).check()


@pytest.mark.parametrize("index8", [False, True])
def test_long_prefix(index8):
    Batch(behind(131072, [700, 5, 3000], 2), [(3, 131072)], 4, 16, page=256, index8=index8).check()


@pytest.mark.parametrize("H,ik_heads", [(1, 0), (2, 0), (8, 0), (8, 1)])
@pytest.mark.parametrize("index8", [False, True])
def test_every_stage_is_used_again(H, ik_heads, index8):
    Batch(behind(262144, [700, 5, 90000], 3) + [(1, 60000)], [(3, 262144)], H, 2, page=256, ik_heads=ik_heads, index8=index8).check()


@pytest.mark.parametrize("index8", [False, True])
def test_the_most_sequences_and_groups(index8):
    Batch([(1 + i % 2, 67 + (i * 37) % 150) for i in range(4096)], [(1, 64)] * 4096, 2, 2, index8=index8).check()


def test_int8_keys_and_values():
    Batch(behind(2048, [0, 100, 63]), [(3, 2048)], 4, 16, index8=True, kv_int8=True).check()


def test_bad_metadata_is_reported():
    bad = msa().ERR_BAD_METADATA
    a = Batch(behind(1280, [20, 100, 64], 2), [(3, 1280)], 2, 16)
    for change in (lambda pb: pb.cache_lens[2].fill_(1281), lambda pb: pb.group_shared[0].fill_(1344),
                   lambda pb: pb.group_starts[1].fill_(4), lambda pb: pb.block_table[0, 2].fill_(1 << 28)):
        keep = a.kw["block_table"].clone()
        pb = a.problem(True)
        change(pb)
        a.run(pb=pb, error=bad)
        a.kw["block_table"].copy_(keep)
    a.check()


def test_a_captured_call_follows_the_metadata():
    m = msa()
    a = Batch(behind(1280, [700, 500, 300], 2), [(3, 1280)], 2, 16)
    pb = a.problem(True)
    ws, out, (sel, nsel) = pb.workspace(), pb.new_out(), pb.new_sel()
    m.forward(pb, a.q, a.iq, a.k, a.v, a.ik, out=out, sel=sel, nsel=nsel, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(pb, a.q, a.iq, a.k, a.v, a.ik, out=out, sel=sel, nsel=nsel, workspace=ws)
    for lens, shared in (([1982, 1782, 1582], 1280), ([1290, 1282, 1400], 1280), ([900, 700, 1500], 640), ([3, 2, 70], 0)):
        pb.cache_lens.copy_(torch.tensor(lens))
        pb.group_shared.fill_(shared)
        graph.replay()
        torch.cuda.synchronize()
        assert m.error_word(ws) == 0
        b = a.problem(False)
        b.cache_lens.copy_(torch.tensor(lens))
        want = a.run(pb=b)
        for x, y in zip((out, sel, nsel), want):
            assert torch.equal(x, y)
