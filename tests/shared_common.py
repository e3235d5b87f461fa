"""Batches whose groups of sequences share a prefix, for the tests of the
dense and the block-sparse attention over them."""
import math

import torch

from dense_common import dense_ref
from gpu_common import msa


def shared_tables(seqs, groups, page, seed=0, spare=2):
    """(block table [B, stride] int32 on the CPU, pages of the pool): pages in any order, those that lie wholly in a
    group's shared positions the same for its sequences."""
    lead, keep, first = list(range(len(seqs))), [0] * len(seqs), 0
    for count, positions in groups:
        for b in range(first + 1, first + count):
            lead[b], keep[b] = first, -(-positions // page)
        first += count
    need = [max(1, -(-L // page)) for _, L in seqs]
    total = sum(max(0, n - k) for n, k in zip(need, keep)) + spare
    ids = torch.randperm(total, generator=torch.Generator().manual_seed(seed))
    table, at = torch.zeros(len(seqs), max(need), dtype=torch.int32), 0
    for b, (n, k) in enumerate(zip(need, keep)):
        k = min(n, k)
        table[b, :k] = table[lead[b], :k]
        table[b, k:n] = ids[at:at + n - k]
        at += n - k
    return table, total


class SharedBatch:
    """Random inputs of one batch with groups [(sequences, positions), ...] and its problem.  `claim` (default: the
    groups) is what the problem is told is shared, which may be fewer positions."""

    def __init__(self, seqs, groups, H, G, page=64, out=torch.bfloat16, int8=False, scale=None, seed=0, spare_rows=0,
                 claim=None, q_gain=2.0, **kw):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.seqs, self.groups, self.H, self.G, self.page, self.out_dtype = seqs, groups, H, G, page, out
        self.table, pages = shared_tables(seqs, groups, page, seed)
        self.table = self.table.cuda()
        self.T = T = pages * page
        self.R = sum(n for n, _ in seqs) + spare_rows
        self.q = (q_gain * torch.randn(self.R, H * G, 128, generator=g, device="cuda")).bfloat16()
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
        self.pb = msa().Problem(H, G, seqs, "cuda", out_dtype=out, cache_tokens=T, scale=self.scale, block_table=self.table,
                                page_size=page, shared=groups if claim is None else claim,
                                num_decode_seqs=len(seqs), num_decode_rows=0, **kw)
        self.pb.total_rows = self.pb.c.total_rows = self.R

    def rows_of(self, b, t):
        return self.table[b].long()[t // self.page] * self.page + t % self.page

    def ref(self):
        bits = 24 if self.out_dtype == torch.float32 else 8
        return dense_ref(self.seqs, self.H, self.G, self.q, self.k, self.v, float(torch.tensor(self.scale)), self.rows_of,
                         self.out_dtype, bits, self.k_scale, self.v_scale)

    def workspace(self):
        ws = self.pb.dense_workspace()
        ws.fill_(0xFF)  # its contents need no initialisation
        return ws

    def run(self, ws=None, out=None, error=0):
        ws = self.workspace() if ws is None else ws
        out = torch.full_like(self.pb.new_out(), float("nan")) if out is None else out
        got = msa().dense_forward(self.pb, self.q, self.k, self.v, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert msa().error_word(ws) == error
        return got

    def check(self, got=None):
        got = self.run() if got is None else got
        ref, bound = self.ref()
        n = sum(c for c, _ in self.seqs)
        err = (got[:n].double() - ref[:n]).abs()
        assert torch.isfinite(got[:n]).all(), "non-finite output"
        worst = (err / bound[:n].clamp_min(1e-300)).max().item()
        assert worst <= 1, f"error {worst:.3g} times its bound"
        if self.out_dtype == torch.float32:
            assert (err.norm() / ref[:n].norm()).item() < 1e-5
        assert torch.isnan(got[n:]).all(), "rows behind the last sequence were written"
        return got
