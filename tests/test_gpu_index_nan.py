"""Index keys that are not finite: a NaN score is passed over in its block's
maximum, and a block of nothing else comes last, the earlier one first.  The
kept blocks against a choice in float64, the outputs against the formula over
them, for every kernel that scores keys: bf16 keys and codes, decode rows,
drafted windows, prompt chunks, groups and the staged calls."""
import math

import pytest
import torch

from gpu_common import msa
from shared_common import shared_tables

pytestmark = pytest.mark.gpu


class Keys:
    """Sequences of `rows` rows each at the given lengths, the first `shared` positions of all of them the same."""

    def __init__(self, rows, lens, codes, shared=0, ik_heads=0, H=2, G=8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.seqs, self.H, self.G, self.codes = [(rows, L) for L in lens], H, G, codes
        groups = [(len(lens), shared)] if shared else []
        table, pages = shared_tables(self.seqs, groups, 64, seed)
        self.table, T, KH = table.cuda(), pages * 64, 1 if ik_heads else H
        self.R = rows * len(lens)
        self.q = torch.randn(self.R, H * G, 128, generator=g, device="cuda").bfloat16()
        self.k, self.v = (torch.randn(T, H, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
        self.iq = torch.randint(-8, 9, (self.R, H, 64), generator=g, device="cuda").bfloat16()
        whole = torch.randint(-127 if codes else -8, 128 if codes else 9, (T, KH, 64), generator=g, device="cuda")
        self.ik = whole.to(torch.int8) if codes else whole.bfloat16()
        self.exp = torch.randint(-5, 2, (T, KH), generator=g, device="cuda").to(torch.int8) if codes else None
        self.kw = dict(block_table=self.table, page_size=64, cache_tokens=T, ik_heads=ik_heads, ik_exp=self.exp, shared=groups or None)

    def spoil(self, b, t, heads=slice(None)):
        """Positions t of sequence b are not finite."""
        rows = self.table[b].long()[t // 64] * 64 + t % 64
        if self.codes:
            x = self.exp[rows]
            x[:, heads] = -128
            self.exp[rows] = x
            y = self.ik[rows]
            y[:, heads] = 0
        else:
            y = self.ik[rows]
            y[:, heads, 17] = float("nan")
        self.ik[rows] = y

    def reference(self):
        """(kept [R, H, 16], outputs [R, H G, 128], their bounds) in float64."""
        kept = torch.full((self.R, self.H, 16), -1, dtype=torch.int32)
        out = torch.zeros(self.R, self.H * self.G, 128, dtype=torch.float64, device="cuda")
        bound, first, scale = torch.zeros_like(out), 0, float(torch.tensor(1 / math.sqrt(128)))
        for b, (n, L) in enumerate(self.seqs):
            t = torch.arange(L, device="cuda")
            rows = self.table[b].long()[t // 64] * 64 + t % 64
            for h in range(self.H):
                key = self.ik[rows, min(h, self.ik.shape[1] - 1)].double()
                if self.codes:
                    e = self.exp[rows, min(h, self.ik.shape[1] - 1)].long()
                    key = key * torch.where(e < -126, math.nan, ((1023 + e) << 52).view(torch.float64))[:, None]
                for i in range(n):
                    p = L - n + i
                    s = torch.nan_to_num(key[:p + 1] @ self.iq[first + i, h].double(), nan=-math.inf, posinf=math.inf, neginf=-math.inf).cpu()
                    m = [s[64 * j:64 * j + 64].max().item() for j in range(p // 64)]
                    best = sorted(sorted(range(len(m)), key=lambda j: (-m[j], j))[:15]) + [p // 64]
                    kept[first + i, h, :len(best)] = torch.tensor(best)
                    at = torch.cat([torch.arange(64 * j, min(64 * j + 64, p + 1), device="cuda") for j in best])
                    q = self.q[first + i, h * self.G:(h + 1) * self.G].double()
                    kk, vv = self.k[rows[at], h].double(), self.v[rows[at], h].double()
                    w = torch.softmax(scale * q @ kk.T, 1)
                    # scores: 128 products summed in fp32 and four roundings; weights: exponentials, two bf16 parts, which the
                    # tensor cores' sums may cut by a unit an addition
                    A = scale * (q.abs() @ kk.abs().T).amax(1)
                    rel = 2 * 132 * 2.0 ** -23 * A + 2.0 ** -22 + 2.0 ** -16 + 2 * len(at) * 2.0 ** -23
                    o = slice(h * self.G, (h + 1) * self.G)
                    out[first + i, o] = w @ vv
                    bound[first + i, o] = (w @ vv.abs()) * rel[:, None] + (w @ vv).abs() * 2.0 ** -24
            first += n
        return kept.cuda(), out, bound

    def check(self, staged=True):
        m = msa()
        pb = m.Problem(self.H, self.G, self.seqs, "cuda", **self.kw)
        ws = pb.workspace()
        ws.fill_(0xFF)
        out, sel, nsel = m.forward(pb, self.q, self.iq, self.k, self.v, self.ik, workspace=ws)
        torch.cuda.synchronize()
        assert m.error_word(ws) == 0
        kept, want, bound = self.reference()
        assert torch.equal(sel, kept)
        assert torch.equal(nsel, (kept >= 0).sum(-1).int())
        assert ((out.double() - want).abs() <= bound).all()
        if staged:
            again = m.select_blocks(pb, m.index_scores(pb, self.iq, self.ik))
            assert torch.equal(again[0], kept) and torch.equal(again[1], nsel)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("rows", [1, 4, 30])
@pytest.mark.parametrize("ik_heads", [0, 1])
@pytest.mark.parametrize("left", [[], [30], [0, 3, 7, 20, 21, 40, 61], list(range(5, 40))])
def test_blocks_without_a_finite_key(rows, codes, ik_heads, left):
    """Of 62 whole blocks those `left` are finite: fewer than the fifteen that a row keeps, or more."""
    a = Keys(rows, [4000], codes, ik_heads=ik_heads)
    for j in range(63):
        if j not in left:
            a.spoil(0, torch.arange(64 * j, min(64 * j + 64, 4000), device="cuda"))
    a.check()


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("rows", [1, 8, 20])
def test_blocks_with_a_few_finite_keys(rows, codes):
    """One finite key a block, anywhere in it, or one that is not."""
    a = Keys(rows, [3000, 1300], codes, seed=rows)
    for b, (_, L) in enumerate(a.seqs):
        for j in range(L // 64):
            t = 64 * j + torch.arange(64, device="cuda")
            one = (7 * j) % 64
            a.spoil(b, t[t % 64 != one] if j % 2 else t[t % 64 == one], slice(None) if j % 3 else slice(0, 1))
    a.check()


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("rows", [1, 3])
def test_blocks_that_a_group_shares(rows, codes):
    a = Keys(rows, [2500, 2100, 2048 + rows], codes, shared=2048, seed=5)
    for j in [0, 1, 5] + list(range(9, 31)):
        a.spoil(0, torch.arange(64 * j, 64 * j + 64, device="cuda"))
    a.spoil(0, torch.arange(2048, 2112, device="cuda"))
    a.spoil(1, torch.arange(2050, 2100 - rows, device="cuda"))
    a.check(staged=False)
