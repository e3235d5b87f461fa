"""The kept blocks for index queries that are no integers.  Keys read back exactly
from codes, but sums are made in 32 bits in another order by every kernel, so
near-ties may be decided differently: each choice is right within the bound of
such a sum, and scores are.

A score is 64 products of bf16 values, exact in 32 bits, added in some order;
an addition rounds, or on the tensor cores cuts, by 2^-23 of the sum at most,
which is at most S = sum_d |q_d k_d|: |error| <= 64 2^-23 S.  The power of two
of a code is exact before the sum and after it."""
import pytest
import torch

from gpu_common import msa
from shared_common import shared_tables

pytestmark = pytest.mark.gpu
EPS = 64 * 2.0 ** -23


def batch(seqs, codes, shared, ik_heads, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    groups = [(len(seqs), shared)] if shared else []
    table, pages = shared_tables(seqs, groups, 64, seed)
    T, KH, R = pages * 64, 1 if ik_heads else H, sum(n for n, _ in seqs)
    q = torch.randn(R, H * 2, 128, generator=g, device="cuda").bfloat16()
    kv = torch.randn(T, H, 128, generator=g, device="cuda").bfloat16()
    iq = torch.randn(R, H, 64, generator=g, device="cuda").bfloat16()
    if codes:
        ik = torch.randn(T, KH, 64, generator=g, device="cuda").mul_(40).round_().clamp_(-127, 127).to(torch.int8)
        exp = torch.randint(-8, -4, (T, KH), generator=g, device="cuda").to(torch.int8)
        values = ik.double() * ((1023 + exp.long()) << 52).view(torch.float64)[..., None]
    else:
        ik, exp = torch.randn(T, KH, 64, generator=g, device="cuda").bfloat16(), None
        values = ik.double()
    pb = msa().Problem(H, 2, seqs, "cuda", block_table=table.cuda(), page_size=64, cache_tokens=T, ik_heads=ik_heads, ik_exp=exp,
                       shared=groups or None)
    return pb, q, iq, kv, ik, values, table.cuda().long()


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("ik_heads", [0, 1])
@pytest.mark.parametrize("H", [1, 4, 8])
@pytest.mark.parametrize("seqs,shared", [([(1, 20000), (1, 5000)], 0), ([(5, 9000), (8, 3000)], 0), ([(300, 9000), (20, 4000)], 0),
                                         ([(1, 9100)] * 9, 8192), ([(4, 5000)] * 3, 4096)])
def test_choices_within_the_sum_s_bound(seqs, shared, H, ik_heads, codes):
    m = msa()
    pb, q, iq, kv, ik, values, table = batch(seqs, codes, shared, ik_heads, H, H + len(seqs))
    _, sel, nsel = m.forward(pb, q, iq, kv, kv, ik)
    scores = m.index_scores(pb, iq, ik)
    first = 0
    for b, (n, L) in enumerate(seqs):
        t = torch.arange(L, device="cuda")
        key = values[table[b][t // 64] * 64 + t % 64].expand(-1, H, -1)
        x = iq[first:first + n].double()
        s = torch.einsum("nhd,thd->nht", x, key)
        S = torch.einsum("nhd,thd->nht", x.abs(), key.abs())
        p = L - n + torch.arange(n, device="cuda")
        seen = (t <= p[:, None])[:, None]
        got = scores[first:first + n, :, :L].double()
        assert ((got - s).abs() <= EPS * S)[seen.expand_as(s)].all()
        blocks = (L - 1) // 64
        cut = lambda y, lowest: y.masked_fill(~seen, lowest)[..., :blocks * 64].reshape(n, H, blocks, 64).amax(-1)  # noqa: E731
        best, slack = cut(s, -float("inf")), cut(EPS * S, 0)
        at = sel[first:first + n].long()
        assert (nsel[first:first + n] == 16).all() and (at.sort(-1).values == at).all() and (at[..., -1] == p[:, None] // 64).all()
        kept = torch.zeros(n, H, blocks + 1, dtype=torch.bool, device="cuda").scatter_(2, at[..., :-1], True)[..., :blocks]
        assert (kept.sum(-1) == 15).all()
        open_ = torch.arange(blocks, device="cuda") < (p // 64)[:, None, None]
        least = (best + slack).masked_fill(~kept, float("inf")).amin(-1)
        most = (best - slack).masked_fill(kept | ~open_, -float("inf")).amax(-1)
        assert (least >= most).all()
        first += n
