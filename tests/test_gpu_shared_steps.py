"""Groups that share a prefix, index keys of 8 bits and the cache writer together, as a server runs them: decoding steps of
a captured graph, graphs that share a workspace, and caches whose offsets pass 32 bits."""
import pytest
import torch

from gpu_common import msa
from shared_common import SharedBatch

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


class Steps(SharedBatch):
    """A batch with an index-key cache of codes.  Index queries and keys are small integers: their codes are exact, and so
    is every score in any order of its sum."""

    def __init__(self, seqs, groups, H, G, **kw):
        probe = SharedBatch(seqs, groups, H, G, **kw)
        self.ik = torch.zeros(probe.T, H, 64, dtype=torch.int8, device="cuda")
        self.exp = torch.zeros(probe.T, H, dtype=torch.int8, device="cuda")
        super().__init__(seqs, groups, H, G, ik_exp=self.exp, **kw)
        g = torch.Generator(device="cuda").manual_seed(9)
        self.ik.copy_(torch.randint(-8, 9, self.ik.shape, generator=g, device="cuda"))
        self.iq = torch.randint(-8, 9, (self.R, H, 64), generator=g, device="cuda").bfloat16()

    def plain(self, seqs):
        """The same batch, at the lengths of `seqs`, without its groups."""
        kw = dict(out_dtype=self.out_dtype, cache_tokens=self.T, scale=self.scale, block_table=self.table, page_size=self.page)
        if self.k_scale is not None:
            kw.update(k_scale=self.k_scale, v_scale=self.v_scale)
        return msa().Problem(self.H, self.G, seqs, "cuda", ik_exp=self.exp, num_decode_seqs=len(seqs), num_decode_rows=0, **kw)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("rows", [1, 3])
def test_decoding_steps(rows, int8):
    """One captured step: the new rows into the caches, the sparse attention, the attention over every position.  Every
    replay sees its rows and lengths: the blocks and outputs are those of a call without groups, and the second output is
    within the bounds of the formula's."""
    m = msa()
    steps = 5
    room = [(rows, 1984 + x + rows * (steps + 1)) for x in (0, 1, 40, 63, 300)] + [(rows, 900 + rows * (steps + 1))]
    a = Steps(room, [(5, 1984)], 4, 8, int8=int8)
    lens = torch.tensor([L - rows * steps for _, L in room])
    g = torch.Generator(device="cuda").manual_seed(3)
    new = {n: torch.empty(a.R, a.H, d, dtype=BF16, device="cuda") for n, d in (("k", 128), ("v", 128), ("ik", 64))}
    ws, dense_ws = a.pb.workspace(), a.workspace()
    out, dense, (sel, nsel) = a.pb.new_out(), a.pb.new_out(), a.pb.new_sel()

    def step():
        m.append_cache(a.pb, new["k"], new["v"], a.k, a.v, new_ik=new["ik"], ik=a.ik, workspace=append_ws)
        m.forward(a.pb, a.q, a.iq, a.k, a.v, a.ik, out=out, sel=sel, nsel=nsel, workspace=ws)
        m.dense_forward(a.pb, a.q, a.k, a.v, out=dense, workspace=dense_ws)

    append_ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    a.pb.cache_lens.copy_(lens)
    for x in new.values():
        x.zero_()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        lens = lens + rows
        a.pb.cache_lens.copy_(lens)
        for n, x in new.items():
            x.copy_(torch.randint(-8, 9, x.shape, generator=g, device="cuda") if n == "ik" else
                    torch.randn(x.shape, generator=g, device="cuda"))
        a.q.copy_(torch.randn(a.q.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert [m.error_word(w) for w in (append_ws, ws, dense_ws)] == [0, 0, 0]
        a.seqs = [(rows, L) for L in lens.tolist()]
        at = torch.cat([a.rows_of(b, torch.arange(L - rows, L, device="cuda")) for b, (_, L) in enumerate(a.seqs)])
        assert torch.equal(torch.ldexp(a.ik[at].float(), a.exp[at][..., None].int()), new["ik"].float())
        want = m.forward(a.plain(a.seqs), a.q, a.iq, a.k, a.v, a.ik)
        for x, y in zip((out, sel, nsel), want):
            assert torch.equal(x, y)
        a.check(dense)


def test_graphs_that_share_a_workspace():
    """Two captured calls of different batches, replayed in turn on one workspace that neither finds as it left it."""
    m = msa()
    a = SharedBatch(behind(4096, [50, 300, 7]), [(3, 4096)], 4, 16, seed=1)
    b = SharedBatch(behind(1024, [500, 30, 70, 64], 4), [(3, 1024)], 4, 16, seed=2, int8=True)
    want = a.run(), b.run()
    ws = torch.empty(max(x.pb.dense_workspace_size() for x in (a, b)), dtype=torch.uint8, device="cuda")
    got, graphs = [torch.zeros_like(x) for x in want], []
    for x, o in zip((a, b), got):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.dense_forward(x.pb, x.q, x.k, x.v, out=o, workspace=ws)
        graphs.append(graph)
    for _ in range(4):
        for graph, o, w in zip(graphs, got, want):
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert m.error_word(ws) == 0
            assert torch.equal(o, w)


def behind(prefix, own, rows=1):
    return [(rows, prefix + x + rows) for x in own]


@pytest.mark.parametrize("int8", [False, True])
def test_offsets_past_32_bits(int8):
    """The pages of a small batch at the end of caches of more than 2^32 elements: the same bits."""
    m = msa()
    seqs = behind(1280, [5, 64, 700], 2) + [(1, 1500)]
    a = Steps(seqs, [(3, 1280)], 8, 4, int8=int8, out=FP32)
    want = a.run(), *m.forward(a.pb, a.q, a.iq, a.k, a.v, a.ik)
    skip = (1 << 32) // (a.H * 128) // a.page + 1  # pages before them
    T = a.T + skip * a.page

    def far(x):
        y = torch.empty(T, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[T - a.T:] = x
        return y

    if int8:
        a.k_scale, a.v_scale = far(a.k_scale), far(a.v_scale)
    # (index keys: 2^31 elements, of one byte)
    a.k, a.v, a.ik, a.exp, a.T, a.table = far(a.k), far(a.v), far(a.ik), far(a.exp), T, a.table + skip
    kw = dict(k_scale=a.k_scale, v_scale=a.v_scale) if int8 else {}
    a.pb = m.Problem(a.H, a.G, seqs, "cuda", out_dtype=FP32, cache_tokens=T, scale=a.scale, block_table=a.table, page_size=a.page,
                     shared=a.groups, num_decode_seqs=len(seqs), num_decode_rows=0, ik_exp=a.exp, **kw)
    got = a.run(), *m.forward(a.pb, a.q, a.iq, a.k, a.v, a.ik)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    new = {n: torch.randn(a.R, a.H, d, device="cuda").bfloat16() for n, d in (("k", 128), ("v", 128), ("ik", 64))}
    m.append_cache(a.pb, new["k"], new["v"], a.k, a.v, new_ik=new["ik"], ik=a.ik)
    at = torch.cat([a.rows_of(b, torch.arange(L - n, L, device="cuda")) for b, (n, L) in enumerate(seqs)])
    for x, scale, y in ((a.k, a.k_scale, new["k"]), (a.v, a.v_scale, new["v"])):
        read = x[at].double() * scale[at][..., None].double() if int8 else x[at].double()
        # bf16 as it is; a code is half a step of its scale, max / 127, off, and the quotient that is rounded some 2^-24 of it
        bound = y.double().abs().amax(-1, keepdim=True) / 127 * (0.5 + 127 * 2.0 ** -22) if int8 else torch.zeros_like(read)
        assert ((read - y.double()).abs() <= bound).all()
    step = ((a.exp[at].long() + 1023) << 52).view(torch.float64)[..., None]  # 2^exp, from its bits
    assert ((a.ik[at].double() * step - new["ik"].double()).abs() <= step / 2).all()


def test_a_bad_page_behind_int8_caches():
    a = SharedBatch(behind(256, [20, 100, 64], 2), [(3, 256)], 2, 16, int8=True)
    a.table[1, 5] = a.T // 64
    a.run(error=msa().binding.ERR_BAD_METADATA)
    a.table[1, 5] = -1
    a.run(error=msa().binding.ERR_BAD_METADATA)
