"""msa_dense_forward with groups of sequences that share a prefix, against a
plain 64-bit implementation, within bounds derived from its roundings
(dense_common.py)."""
import pytest
import torch

from gpu_common import msa
from shared_common import SharedBatch

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def behind(prefix, own, rows=1):
    """Sequences behind a prefix: `own` positions each before their rows' own."""
    return [(rows, prefix + x + rows) for x in own]


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("prefix", [64, 128, 192, 1024])
def test_one_group(prefix, out):
    SharedBatch(behind(prefix, [0, 1, 63, 64, 65, 200]), [(6, prefix)], 2, 16, out=out).check()


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("own", [[0], [1], [62], [63], [64], [127, 128], [129, 0], [191, 193, 255, 256, 257]])
def test_own_positions_at_tile_edges(own, out):
    SharedBatch(behind(192, own), [(len(own), 192)], 1, 16, out=out, seed=len(own) + own[0]).check()


@pytest.mark.parametrize("H,G", [(1, 1), (2, 3), (4, 5), (8, 7), (8, 1), (4, 8), (1, 13), (1, 16), (2, 9)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_head_layouts(H, G, out):
    seqs = behind(320, [5, 0, 77], 3) + behind(64, [9, 300], 1) + [(1, 1), (2, 130)]
    SharedBatch(seqs, [(3, 320), (2, 64)], H, G, out=out, seed=H * G).check()


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_windows(rows, out):
    SharedBatch(behind(448, [0, 3, 64, 150, 700], rows), [(5, 448)], 2, 16, page=64, out=out, seed=rows).check()


@pytest.mark.parametrize("count", [2, 7, 8, 9, 16, 17, 33, 70])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_rows_of_a_group_over_tiles(count, out):
    """One M tile holds 8 rows of 16 heads, an item two of them."""
    SharedBatch(behind(640, [(37 * i) % 150 for i in range(count)]), [(count, 640)], 2, 16, out=out, seed=count).check()


def test_uneven_rows_and_a_sequence_without_any():
    seqs = [(1, 300), (0, 257), (8, 264), (3, 261), (0, 400), (5, 900), (1, 1), (0, 64), (4, 77)]
    SharedBatch(seqs, [(6, 256)], 2, 16, spare_rows=5).check()


def test_all_sequences_of_a_group_without_rows():
    SharedBatch([(0, 300), (0, 400), (1, 500), (2, 90)], [(2, 256), (1, 192)], 4, 4, spare_rows=3).check()


@pytest.mark.parametrize("claim", [1, 63, 64, 100, 191, 256, 301])
def test_shared_positions_of_any_number(claim):
    """Whole blocks of what is said to be shared are; the rest is read for each sequence."""
    SharedBatch(behind(320, [0, 40, 90], 2), [(3, 320)], 2, 8, claim=[(3, claim)], seed=claim).check()


def test_groups_without_shared_positions():
    SharedBatch(behind(0, [5, 100, 300]) + [(1, 10)], [(3, 0)], 2, 8).check()


def test_one_sequence_groups():
    SharedBatch(behind(256, [9]) + behind(128, [70]) + behind(0, [700]), [(1, 256), (1, 128)], 2, 8).check()


def test_same_as_without_groups():
    a = SharedBatch(behind(1024, [5, 100, 300, 17]), [(4, 1024)], 4, 16, out=FP32)
    with_groups = a.run()
    a.pb.c.num_groups = 0
    without = a.run()
    # both within 1e-5 of the formula in the 2-norm
    assert ((with_groups - without).norm() / without.norm()).item() < 2e-5


@pytest.mark.parametrize("page", [64, 128, 512, 4096])
def test_pages(page):
    SharedBatch(behind(4096, [1, 4095, 30]), [(3, 4096)], 2, 8, page=page).check()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_keys_of_more_than_one_part(out):
    """Parts end after 32,768 keys, of the prefix and of a sequence's own."""
    SharedBatch(behind(66048, [40000, 1, 32768, 700], 2), [(4, 66048)], 1, 16, page=256, out=out).check()


def test_no_drift_over_long_contexts():
    """Equal keys and values: the output is the value itself whatever the length; one cut in the same direction an
    addition would show.  Bound: half a step of bf16 and the weights' roundings, 2^-9 and 2^-8."""
    a = SharedBatch(behind(131072, [3000, 5]), [(2, 131072)], 1, 16, page=4096)
    a.k.fill_(0.5)
    a.v.fill_(1.25)
    got = a.run().double()
    assert ((got - 1.25).abs().max() / 1.25).item() <= 2.0 ** -8


def test_many_sequences_and_groups():
    """More entries than the block-wide scan takes at a time."""
    groups = [(3, 64 * (1 + i % 3)) for i in range(150)]
    seqs = [s for count, p in groups for s in behind(p, [(p * 7 + j * 31) % 90 for j in range(count)])]
    seqs += [(1, 1 + (i * 13) % 200) for i in range(50)]
    SharedBatch(seqs, groups, 1, 4).check()


def test_a_thousand_samples_of_one_prompt():
    SharedBatch(behind(512, [(i * 29) % 64 for i in range(1000)]), [(1000, 512)], 1, 4).check()


@pytest.mark.parametrize("int8", [False, True])
def test_the_most_sequences_and_groups(int8):
    SharedBatch([(1 + i % 2, 67 + (i * 37) % 150) for i in range(4096)], [(1, 64)] * 4096, 1, 2, int8=int8).check()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_tokens_that_a_row_does_not_see(out):
    """Positions past a sequence's length, and its later tokens, may hold NaN or infinities."""
    a = SharedBatch(behind(256, [0, 30, 64, 100], 4), [(4, 256)], 2, 16, out=out)
    ref, bound = a.ref()
    seen = torch.zeros(a.T, dtype=torch.bool, device="cuda")
    for b, (n, L) in enumerate(a.seqs):
        seen[a.rows_of(b, torch.arange(L, device="cuda"))] = True
    for bad in (float("nan"), float("inf")):
        a.k[~seen], a.v[~seen] = bad, bad
        got = a.run()
        assert ((got.double() - ref).abs() <= bound).all()
    # each sequence's last token: its last row alone meets it
    for b, (n, L) in enumerate(a.seqs):
        last = a.rows_of(b, torch.tensor([L - 1], device="cuda"))
        a.v[last] = float("nan")
        a.k[last] = float("inf")
    got = a.run()
    err = (got.double() - ref).abs() <= bound
    keep = torch.arange(a.R, device="cuda") % 4 != 3
    assert err[keep].all()
    assert torch.isnan(got[~keep]).any(-1).all()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_large_and_small_scores(out):
    """The maximum rises late and far (prefix small, own keys large) and early."""
    a = SharedBatch(behind(512, [200, 64, 5]), [(3, 512)], 2, 16, out=out, q_gain=6.0)
    a.k[a.rows_of(0, torch.arange(400, 500, device="cuda"))] *= 4
    a.k[a.rows_of(1, torch.arange(530, 560, device="cuda"))] *= 8
    a.check()


@pytest.mark.parametrize("scale", [0.0, 1e-3, 1.0])
def test_scales(scale):
    SharedBatch(behind(256, [10, 300]), [(2, 256)], 2, 8, out=FP32, scale=scale, q_gain=0.5).check()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_int8_caches(out):
    seqs = behind(640, [0, 1, 63, 200], 1) + behind(128, [5, 300], 4) + [(1, 1), (2, 700)]
    SharedBatch(seqs, [(4, 640), (2, 128)], 2, 16, out=out, int8=True).check()


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (4, 16)])
def test_int8_caches_over_many_tiles(H, G, out):
    """Groups of one M tile, of two and of an odd number, prefixes that end inside a tile of 128 keys, own positions of any
    length: every ring slot and scale slot is used again."""
    rows = 128 // G
    most = min(8, rows)
    groups, seqs = [], []
    for tiles, S in ((1, 1984), (2, 2112), (3, 1280)):
        n = min(rows * tiles // most + (tiles > 1), 40)
        seqs += behind(S, [(37 * i) % 700 for i in range(n)], most)
        groups.append((n, S))
    SharedBatch(seqs + [(most, 1500), (1, 130)], groups, H, G, out=out, int8=True, seed=3).check()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_int8_parts_of_a_long_prefix(out):
    SharedBatch(behind(40000, [0, 100, 33000], 1), [(3, 40000)], 1, 16, out=out, int8=True).check()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_int8_scales_past_the_end_do_not_matter(out):
    a = SharedBatch(behind(256, [1, 70, 129, 190], 1) + [(1, 3)], [(4, 256)], 2, 16, out=out, int8=True)
    used = torch.zeros(a.T, dtype=torch.bool, device="cuda")
    for b, (n, L) in enumerate(a.seqs):
        used[a.rows_of(b, torch.arange(L, device="cuda"))] = True
    a.k_scale[~used] = float("nan")
    a.v_scale[~used] = float("inf")
    a.check()


def test_the_same_call_gives_the_same_bits():
    a = SharedBatch(behind(8192, [100 * i for i in range(20)], 2), [(20, 8192)], 4, 16)
    first, ws = a.run(), a.workspace()
    for _ in range(3):
        assert torch.equal(a.run(ws), first)


def test_a_captured_call_follows_the_metadata():
    """cache_lens, the block table and the groups are read by the kernels: a replay sees what they hold then."""
    m = msa()
    long = SharedBatch(behind(1024, [500, 300, 100], 2), [(3, 1024)], 2, 16)
    ws, out = long.workspace(), torch.zeros_like(long.pb.new_out())
    m.dense_forward(long.pb, long.q, long.k, long.v, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.dense_forward(long.pb, long.q, long.k, long.v, out=out, workspace=ws)
    for lens, shared in (([1526, 1326, 1126], 1024), ([1030, 1026, 1100], 1024), ([900, 700, 1500], 640), ([3, 2, 70], 0)):
        long.pb.cache_lens.copy_(torch.tensor(lens))
        long.pb.group_shared.fill_(shared)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert m.error_word(ws) == 0
        long.seqs = [(2, L) for L in lens]
        long.check(out)


def test_two_streams_at_once():
    a = SharedBatch(behind(4096, [50, 300, 7]), [(3, 4096)], 4, 16, seed=1)
    b = SharedBatch(behind(2048, [500, 30], 4), [(2, 2048)], 4, 16, seed=2)
    want = a.run(), b.run()
    ws = a.workspace(), b.workspace()
    got = [torch.empty_like(x) for x in want]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        for x, w, s, o in zip((a, b), ws, streams, got):
            with torch.cuda.stream(s):
                msa().dense_forward(x.pb, x.q, x.k, x.v, out=o, workspace=w)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_bad_metadata_is_reported():
    m = msa()

    def batch():
        return SharedBatch(behind(256, [20, 100, 64], 2), [(3, 256)], 2, 16)

    def spoiled(change):
        a = batch()
        change(a)
        a.run(error=m.binding.ERR_BAD_METADATA)

    spoiled(lambda a: a.table[0, 1].fill_(a.T // 64))        # a page outside the pool, of the prefix
    spoiled(lambda a: a.table[1, 5].fill_(-1))               # of a sequence's own
    spoiled(lambda a: a.pb.block_table[1].fill_(1 << 30))
    spoiled(lambda a: a.pb.cache_lens[2].fill_(257))         # rows before the end of the shared positions
    spoiled(lambda a: a.pb.cache_lens[2].fill_(1 << 20))     # past max_cache_len
    spoiled(lambda a: a.pb.group_shared[0].fill_(320))       # more than the host's bound
    spoiled(lambda a: a.pb.group_shared[0].fill_(-64))
    spoiled(lambda a: a.pb.group_starts[1].fill_(4))         # more sequences than there are
    spoiled(lambda a: a.pb.group_starts.copy_(torch.tensor([2, 1], dtype=torch.int32)))
    a = batch()
    a.pb.c.max_group_rows = 5                                # fewer than the group has
    a.run(error=m.binding.ERR_BAD_METADATA)
    a.pb.c.max_group_rows = 6
    a.check()
