"""msa_dense_forward against a plain 64-bit implementation, within bounds
derived from its roundings (dense_common.py)."""
import math

import pytest
import torch

from dense_common import dense_ref
from gpu_common import msa

pytestmark = pytest.mark.gpu


class Batch:
    """Random inputs of one batch and its problem."""

    def __init__(self, seqs, H, G, int8=False, page=0, out=torch.bfloat16, scale=None, seed=0, spare_rows=0, q_gain=2.0,
                 lead=5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        m = msa()
        self.seqs, self.H, self.G, self.out_dtype, self.int8 = seqs, H, G, out, int8
        R = sum(n for n, _ in seqs) + spare_rows
        B = len(seqs)
        self.starts = self.table = None
        kw = {}
        if page:
            need = [max(1, -(-L // page)) for _, L in seqs]
            ids = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(seed))
            self.table = torch.zeros(B, max(need), dtype=torch.int32)
            at = 0
            for b, c in enumerate(need):
                self.table[b, :c] = ids[at:at + c]
                at += c
            T = (sum(need) + 2) * page
            self.table = self.table.cuda()
            kw.update(block_table=self.table, page_size=page)
        else:
            self.starts, at = [], lead
            for _, L in seqs:
                self.starts.append(at)
                at += L + 3
            T = at
            kw.update(cache_starts=self.starts)
        self.page, self.T = page, T
        self.q = (q_gain * torch.randn(R, H * G, 128, generator=g, device="cuda")).bfloat16()
        self.k_scale = self.v_scale = None
        if int8:
            self.k = torch.randint(-127, 128, (T, H, 128), generator=g, device="cuda", dtype=torch.int8)
            self.v = torch.randint(-127, 128, (T, H, 128), generator=g, device="cuda", dtype=torch.int8)
            self.k_scale = (0.5 + torch.rand(T, H, generator=g, device="cuda")) / 64
            self.v_scale = (0.5 + torch.rand(T, H, generator=g, device="cuda")) / 64
            kw.update(k_scale=self.k_scale, v_scale=self.v_scale)
        else:
            self.k = torch.randn(T, H, 128, generator=g, device="cuda").bfloat16()
            self.v = (torch.randn(T, H, 128, generator=g, device="cuda") + 0.3).bfloat16()
        self.scale = 1 / math.sqrt(128) if scale is None else scale
        # the host rows per sequence drive the bounds; a sequence of no rows still has a cache
        self.pb = m.Problem(H, G, seqs, "cuda", out_dtype=out, cache_tokens=T, scale=self.scale,
                            num_decode_seqs=-1 if any(n == 0 for n, _ in seqs) else "auto", **kw) \
            if not spare_rows else self._spare(m, R, kw)

    def _spare(self, m, R, kw):
        pb = m.Problem(self.H, self.G, self.seqs, "cuda", out_dtype=self.out_dtype, cache_tokens=self.T,
                       scale=self.scale, **kw)
        pb.total_rows = R
        pb.c.total_rows = R
        return pb

    def rows_of(self, b, t):
        if self.table is not None:
            return self.table[b].long()[t // self.page] * self.page + t % self.page
        return self.starts[b] + t

    def ref(self):
        weight_bits = 24 if self.out_dtype == torch.float32 else 8
        return dense_ref(self.seqs, self.H, self.G, self.q, self.k, self.v, float(torch.tensor(self.scale)), self.rows_of,
                         self.out_dtype, weight_bits, self.k_scale, self.v_scale)

    def dirty_workspace(self):
        ws = self.pb.dense_workspace()
        ws.fill_(0xFF)  # its contents need no initialisation
        return ws

    def run(self, ws=None, out=None):
        ws = self.dirty_workspace() if ws is None else ws
        out = torch.full_like(self.pb.new_out(), float("nan")) if out is None else out
        got = msa().dense_forward(self.pb, self.q, self.k, self.v, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert msa().error_word(ws) == 0
        return got

    def check(self, got=None):
        got = self.run() if got is None else got
        ref, bound = self.ref()
        n = sum(c for c, _ in self.seqs)
        err = (got[:n].double() - ref[:n]).abs()
        assert torch.isfinite(got[:n]).all(), "non-finite output"
        worst = (err / bound[:n].clamp_min(1e-300)).max().item()  # a value of 0 has no error and no bound
        assert worst <= 1, f"error {worst:.3g} times its bound"
        if self.out_dtype == torch.float32:  # the sums above are worst cases: in the 2-norm fp32 outputs are near fp32
            assert (err.norm() / ref[:n].norm()).item() < 1e-5


EDGES = [1, 2, 15, 63, 64, 65, 127, 128, 129, 191, 193, 500]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_single_rows_at_block_edges(out, page, int8):
    Batch([(1, L) for L in EDGES], 2, 16, int8, page, out).check()


@pytest.mark.parametrize("H,G", [(1, 1), (2, 3), (4, 5), (8, 7), (8, 1), (4, 8), (1, 13), (1, 16)])
@pytest.mark.parametrize("int8", [False, True])
def test_head_layouts_single_rows(H, G, int8):
    Batch([(1, 700), (1, 1), (1, 333)], H, G, int8, 128, torch.float32, seed=H * G).check()


@pytest.mark.parametrize("n", [2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("G", [1, 4, 16])
def test_drafted_windows(n, G):
    Batch([(n, L) for L in (n, n + 1, 64, 130, 777)], 2, G, n % 2 == 1, 64 if n > 4 else 0,
          torch.bfloat16 if n % 3 else torch.float32, seed=n).check()


@pytest.mark.parametrize("n", [9, 16, 17, 63, 64, 65, 127, 129, 260])
@pytest.mark.parametrize("G", [1, 6, 16])
def test_prompts_without_prefix(n, G):
    Batch([(n, n)], 2, G, n % 2 == 0, 0 if n % 4 else 64, torch.float32 if G == 6 else torch.bfloat16, seed=n).check()


@pytest.mark.parametrize("L", [300, 319, 320, 321, 384, 385, 1000])
def test_prompts_behind_a_prefix(L):
    for G in (5, 16):
        for int8 in (False, True):
            Batch([(70, L)], 1, G, int8, 64, torch.bfloat16, seed=L).check()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("int8", [False, True])
def test_packed_sequences_of_every_kind(out, int8):
    seqs = [(1, 1), (130, 130), (1, 900), (9, 9), (33, 400), (4, 70), (200, 201), (8, 8), (1, 64), (16, 2000)]
    Batch(seqs, 4, 6, int8, 128, out, seed=3).check()
    Batch(seqs, 2, 16, int8, 0, out, seed=4).check()


@pytest.mark.parametrize("seqs", [[(1, 40000)], [(1, 33333), (1, 5)], [(4, 30001)], [(64, 20011)]])
def test_long_contexts_are_split(seqs):
    for int8 in (False, True):
        Batch(seqs, 1, 16, int8, 64, torch.float32, seed=7).check()


def test_many_sequences():
    Batch([(1, 1 + (37 * i) % 200) for i in range(700)], 1, 4, False, 64, torch.bfloat16).check()
    Batch([(1 + i % 12, 20 + (37 * i) % 200) for i in range(300)], 2, 3, True, 64, torch.bfloat16).check()


@pytest.mark.parametrize("count", [2, 12, 40, 130, 150, 255, 256, 300])
@pytest.mark.parametrize("H,int8", [(1, False), (8, False), (4, True)])
def test_any_number_of_single_rows(count, H, int8):
    """Shares that begin and end inside sequences, hold several, or hold none."""
    Batch([(1, 1 + (7919 * i) % (64 if i % 3 else 2000)) for i in range(count)], H, 4, int8, 64,
          torch.float32 if count % 4 else torch.bfloat16, seed=count).check()


@pytest.mark.parametrize("seqs", [[(8, 900), (1, 64), (8, 8)], [(5, 20000), (8, 3000)], [(8, 70 + i) for i in range(90)]])
def test_several_tiles_of_rows_a_sequence(seqs):
    for int8 in (False, True):  # (G = 2: one tile; 16 with an int8 cache: up to eight)
        for G in (2, 16):
            Batch(seqs, 2, G, int8, 64, torch.float32, seed=G).check()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("G", [6, 16])
def test_decodes_windows_and_prompts_in_one_call(G, int8, out):
    """Contexts long enough that each kind runs in its own kernel."""
    seqs = [(1, 5000), (40, 4200), (1, 70), (4, 4500), (8, 8), (12, 12), (5, 300), (200, 700)]
    Batch(seqs, 2, G, int8, 64, out, seed=G).check()


@pytest.mark.parametrize("int8", [False, True])
def test_many_sequences_of_every_kind(int8):
    seqs = [((1, 4, 12, 7, 20)[i % 5], 20 + (37 * i) % 200) for i in range(450)]
    Batch(seqs, 1, 8, int8, 64, torch.bfloat16).check()
    seqs[17] = (12, 5000)  # (every kind in its own kernel)
    Batch(seqs, 1, 8, int8, 0, torch.float32).check()
    Batch(seqs[:40], 4, 8, int8, 0, torch.bfloat16).check()


@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("int8", [False, True])
def test_cache_rows_beyond_32_bit_offsets(n, int8):
    """Rows from 4,200,000 on of 8 heads of 128 values: elements past 2^32."""
    Batch([(n, 300), (n, 77)], 8, 4, int8, 0, torch.float32, lead=4_200_000).check()


def test_int8_prompts_widened_a_few_at_a_time():
    """The widened copy of a 2^20-token context and its neighbours is larger than one pass may hold."""
    Batch([(40, 50), (9, 1 << 20), (1, 300), (130, 130)], 8, 1, True, 0, torch.bfloat16).check()
    Batch([(40, 50), (9, 1 << 20), (20, 70)], 8, 1, True, 0, torch.float32).check()


def test_sequences_may_share_pages():
    for n in (1, 4, 40):
        b = Batch([(n, 300), (n, 300), (n, 300)], 2, 8, n == 4, 64)
        b.table[1, :3] = b.table[0, :3]  # a common prefix
        b.table[2] = b.table[0]
        b.check()


def test_two_calls_at_once_on_two_streams():
    m = msa()
    batches = [Batch([(300, 6000)], 2, 16), Batch([(1, 30000), (4, 9000)], 2, 16), Batch([(64, 5000)], 2, 16, True)]
    want = [b.run() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    got = [[] for _ in batches]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s, g in zip(batches, streams, got):
            with torch.cuda.stream(s):
                g.append(m.dense_forward(b.pb, b.q, b.k, b.v))  # (a workspace of its own)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("scale,gain", [(0.0, 2.0), (4.0, 3.0), (1e-3, 1.0)])
def test_flat_and_peaked_softmax(n, scale, gain):
    Batch([(n, 500), (n, 65)], 2, 16, False, 0, torch.bfloat16, scale=scale, q_gain=gain).check()


@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("page", [0, 64])
def test_cache_rows_past_the_length_may_hold_anything(n, int8, page):
    """NaN and infinities wherever no position of a sequence lies."""
    b = Batch([(n, 70), (n, 300), (n, n), (n, 128)], 2, 16, int8, page, torch.bfloat16, seed=n)
    used = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    for i, (_, L) in enumerate(b.seqs):
        used[b.rows_of(i, torch.arange(L, device="cuda"))] = True
    if int8:
        b.k_scale[~used] = float("nan")
        b.v_scale[~used] = float("inf")
    else:
        b.k[~used] = float("nan")
        b.v[~used] = float("inf")
    b.check()


@pytest.mark.parametrize("n", [3, 40])
def test_later_tokens_do_not_reach_earlier_rows(n):
    """A NaN or an infinity in the key and value of a later token of the same chunk."""
    b = Batch([(n, 200)], 2, 16, False, 0, torch.bfloat16, seed=1)
    # a spoiled row is computed again in another order of the same operations, with fp32 weights, so it stays within
    # the bound of the formula (which allows bf16 weights) rather than the same bits
    ref, bound = b.ref()
    at = n - 2
    row = b.rows_of(0, torch.tensor(200 - n + at)).item()
    for key, value in ((float("nan"), float("nan")), (0, float("inf")), (0, -float("inf"))):
        b.k[row], b.v[row] = key, value
        after = b.run()
        assert ((after[:at].double() - ref[:at]).abs() <= bound[:at]).all()
        assert not torch.isfinite(after[at:]).any()


@pytest.mark.parametrize("n", [1, 5, 40, 200])
def test_int8_scales_of_any_size(n):
    """Scales that differ by 2^-12 from token to token, blocks of zero, tiny and huge scales."""
    b = Batch([(n, 500), (n, 1000)], 2, 16, True, 64, torch.bfloat16, seed=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    b.pb.v_scale.mul_(2.0 ** torch.randint(-12, 1, b.v_scale.shape, generator=g, device="cuda"))
    b.pb.k_scale.mul_(2.0 ** torch.randint(-6, 1, b.k_scale.shape, generator=g, device="cuda"))
    for seq in range(2):
        rows = b.rows_of(seq, torch.arange(500, device="cuda"))
        b.pb.v_scale[rows[64:128]] = 0
        b.pb.v_scale[rows[130:200]] *= 2.0 ** -60
        b.pb.k_scale[rows[256:320]] = 0
        b.pb.v_scale[rows[320:384], 0] *= 2.0 ** 40
        b.pb.k_scale[rows[200:250]] *= 2.0 ** -100
    b.k_scale, b.v_scale = b.pb.k_scale, b.pb.v_scale
    b.check()
    b.pb.v_scale.mul_(2.0 ** -100)
    b.check()
    b.pb.v_scale.mul_(2.0 ** 100).mul_(2.0 ** 60)
    b.check()


@pytest.mark.parametrize("n", [3, 40])
def test_int8_later_tokens_do_not_reach_earlier_rows(n):
    b = Batch([(n, 200)], 2, 16, True, 0, torch.bfloat16, seed=1)
    ref, bound = b.ref()
    at = n - 2
    row = b.rows_of(0, torch.tensor(200 - n + at)).item()
    for ks, vs in ((float("nan"), float("nan")), (0.01, float("inf")), (float("inf"), 0.01)):
        b.pb.k_scale[row], b.pb.v_scale[row] = ks, vs
        after = b.run()
        assert ((after[:at].double() - ref[:at]).abs() <= bound[:at]).all()
        if ks != float("inf"):  # (an infinite key scale makes a score of either sign: weight 0, or a NaN)
            assert not torch.isfinite(after[at:]).all(-1).any()


@pytest.mark.parametrize("n", [1, 4, 40, 300])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_values_and_queries_that_are_not_finite_stay_where_they_belong(n, out):
    b = Batch([(n, 400), (n, 333)], 2, 16, False, 64, out, seed=3)
    ref, bound = b.ref()
    rows = b.rows_of(0, torch.arange(400, device="cuda"))
    b.v[rows[50], 1, 7] = float("inf")  # seen by every row of sequence 0: one value of head 1's outputs
    b.q[n // 2, 3] = float("nan")       # a query head of one row: all of it
    got = b.run()
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[:n, 16:, 7] = True
    bad[n // 2, 3] = True
    assert not torch.isfinite(got[bad]).any()
    assert ((got.double() - ref).abs() <= bound)[~bad].all()


@pytest.mark.parametrize("n", [40, 4])
def test_many_rows_that_are_not_finite_over_a_long_context(n):
    """Nothing is computed twice for them, and a value that only some rows of a chunk see is still told apart."""
    b = Batch([(n, 1 << 19), (n, 333)], 1, 16, False, 0, torch.bfloat16, seed=3)
    rows = b.rows_of(0, torch.arange(1 << 19, device="cuda"))
    b.q[: n // 2] = float("nan")
    b.v[rows[100], 0, 5] = float("nan")
    got = b.run()
    assert not torch.isfinite(got[: n // 2]).any() and not torch.isfinite(got[:n, :, 5]).any()
    b.q[:n] = torch.randn(n, 16, 128, device="cuda").bfloat16()
    b.v[rows[100], 0, 5] = 0
    ref, bound = b.ref()  # (before the infinity, which the plain form would multiply by weights of zero)
    b.v[rows[(1 << 19) - 2], 0, 9] = float("inf")  # the last two rows see it
    got = b.run()
    assert ((got[: n - 2].double() - ref[: n - 2]).abs() <= bound[: n - 2]).all()
    assert not torch.isfinite(got[n - 2 : n, :, 9]).any()
    assert ((got[n:].double() - ref[n:]).abs() <= bound[n:]).all()


def test_rows_behind_the_last_sequence_stay():
    for seqs in ([(1, 100), (1, 30)], [(20, 100), (5, 30)], [(4, 100)]):
        b = Batch(seqs, 2, 8, spare_rows=7)
        out = torch.full_like(b.pb.new_out(), 7.0)
        b.check(b.run(out=out))
        assert (out[sum(n for n, _ in seqs):] == 7).all()


def test_sequences_of_no_rows_are_skipped():
    m = msa()
    b = Batch([(1, 100), (3, 30), (20, 90)], 2, 8)
    # the same rows as sequences 0, 2 and 4 of a batch whose sequences 1 and 3 have none
    pb = m.Problem(2, 8, [(1, 100), (1, 1), (3, 30), (1, 1), (20, 90)], "cuda", out_dtype=torch.bfloat16,
                   cache_tokens=b.T, cache_starts=[b.starts[0], 0, b.starts[1], 0, b.starts[2]], num_decode_seqs=-1)
    pb.cu_rows.copy_(torch.tensor([0, 1, 1, 4, 4, 24], dtype=torch.int32))
    pb.c.total_rows = pb.total_rows = 24
    pb.c.num_decode_rows = 0
    ws = pb.dense_workspace()
    got = m.dense_forward(pb, b.q, b.k, b.v, workspace=ws)
    torch.cuda.synchronize()
    assert m.error_word(ws) == 0
    assert torch.equal(got, b.run()) or b.check(got) is None


def test_bad_metadata_is_reported_and_contained():
    m = msa()
    for n in (1, 4, 40):
        b = Batch([(n, 300), (n, 200)], 2, 16, page=64)
        good = b.run()
        for what in ("page", "length"):
            saved = b.table.clone(), b.pb.cache_lens.clone()
            if what == "page":
                b.pb.block_table[0, 1] = b.T // 64 + 5
            else:
                b.pb.cache_lens[0] = 300 + 64 * 100
            ws = b.dirty_workspace()
            out = m.dense_forward(b.pb, b.q, b.k, b.v, workspace=ws)
            torch.cuda.synchronize()
            assert m.error_word(ws) == m.ERR_BAD_METADATA
            assert torch.isfinite(out[n:]).all()
            assert (out[n:].double() - good[n:].double()).abs().max() < 0.05  # the other sequence is untouched by it
            b.pb.block_table.copy_(saved[0])
            b.pb.cache_lens.copy_(saved[1])


@pytest.mark.parametrize("seqs", [[(1, 5000), (1, 70)], [(4, 3000)], [(300, 700), (1, 900)]])
def test_repeated_calls_and_graph_replays_agree(seqs):
    """The same bits every time: eagerly, from a captured graph, on another
    stream, and with a workspace that another graph used in between."""
    m = msa()
    b = Batch(seqs, 2, 16, False, 64, torch.bfloat16)
    c = Batch([(1, 900), (40, 333)], 2, 16, True, 0, torch.bfloat16)
    first, other = b.run(), c.run()
    ws = torch.empty(max(b.pb.dense_workspace_size(), c.pb.dense_workspace_size()), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(first), torch.empty_like(other)]
    graphs = []
    for x, out in zip((b, c), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.dense_forward(x.pb, x.q, x.k, x.v, out=out, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], other)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = m.dense_forward(b.pb, b.q, b.k, b.v)
    same = m.dense_forward(c.pb, c.q, c.k, c.v)
    torch.cuda.synchronize()
    assert torch.equal(again, first) and torch.equal(same, other)


def test_agrees_with_the_sparse_attention_where_every_block_is_kept():
    m = msa()
    b = Batch([(1, 1000), (3, 900), (50, 1024)], 4, 16, out=torch.float32)
    iq = torch.randn(b.pb.total_rows, 4, 64, device="cuda").bfloat16()
    ik = torch.randn(b.T, 4, 64, device="cuda").bfloat16()
    sparse, _, _ = m.forward(b.pb, b.q, iq, b.k, b.v, ik)
    dense = b.run()
    # the sparse kernels carry the weights as two bf16 parts (2^-16) and state 2e-3
    assert (sparse - dense).abs().max() < 1e-3


def test_wrong_arguments_are_refused():
    m = msa()
    b = Batch([(1, 100)], 2, 4)
    with pytest.raises(TypeError):
        m.dense_forward(b.pb, b.q.float(), b.k, b.v)
    with pytest.raises(ValueError):
        m.dense_forward(b.pb, b.q, b.k[:-1], b.v)
    with pytest.raises(ValueError):
        m.dense_forward(b.pb, b.q.cpu(), b.k, b.v)
    with pytest.raises(m.MsaError):
        m.dense_forward(b.pb, b.q, b.k, b.v, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        m.dense_forward(b.pb, b.q, b.k, b.v, out=torch.empty(1, 8, 128, device="cuda"))
