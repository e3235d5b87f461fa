"""Index keys of 8 bits: written by msa_append_cache, read by
msa_index_scores and msa_forward (decode rows, drafted windows, prompt chunks,
mixed batches).  A code times its power of two is a bf16 value exactly, so a
forward over codes has to choose the very blocks, and give the very outputs,
that it gives over a bf16 cache of the same values.  Index queries and codes
are small integers here: their scores are exact in fp32 in any order."""
import math

import pytest
import torch

from dense_common import rotate_ref
from gpu_common import msa

pytestmark = pytest.mark.gpu


def paged(seqs, page, seed=0):
    need = [max(1, -(-L // page)) for _, L in seqs]
    ids = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(seed))
    table, at = torch.zeros(len(seqs), max(need), dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table.cuda(), (sum(need) + 2) * page


class Sparse:
    """Inputs of one forward; `both()` runs it over codes and over the bf16 values that they stand for."""

    def __init__(self, seqs, H, G, page=0, ik_heads=0, kv_int8=False, seed=0, out=torch.float32, exps=(-7, 3), lead=3, **kw):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.seqs, self.H, self.G = seqs, H, G
        if page:
            table, T = paged(seqs, page, seed)
            kw.update(block_table=table, page_size=page)
        else:
            starts, T = [], lead
            for _, L in seqs:
                starts.append(T)
                T += L + 1
            kw.update(cache_starts=starts)
        KH = 1 if ik_heads == 1 else H
        R = sum(n for n, _ in seqs)
        ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda")  # noqa: E731
        self.q = torch.randn(R, H * G, 128, generator=g, device="cuda").bfloat16()
        self.iq = ints(-8, 9, R, H, 64).bfloat16()
        self.codes = ints(-127, 128, T, KH, 64).to(torch.int8)
        self.exp = ints(exps[0], exps[1] + 1, T, KH).to(torch.int8)
        if kv_int8:
            self.k, self.v = (ints(-127, 128, T, H, 128).to(torch.int8) for _ in range(2))
            kw.update(k_scale=0.01 + torch.rand(T, H, generator=g, device="cuda") / 64,
                      v_scale=0.01 + torch.rand(T, H, generator=g, device="cuda") / 64)
        else:
            self.k, self.v = (torch.randn(T, H, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
        self.kw = dict(out_dtype=out, cache_tokens=T, ik_heads=ik_heads, **kw)

    def values(self):
        return torch.ldexp(self.codes.float(), self.exp[..., None].int()).bfloat16()

    def run(self, ik, **kw):
        m = msa()
        pb = m.Problem(self.H, self.G, self.seqs, "cuda", **self.kw, **kw)
        ws = pb.workspace()
        ws.fill_(0xFF)
        out = torch.full_like(pb.new_out(), float("nan"))
        out, sel, nsel = m.forward(pb, self.q, self.iq, self.k, self.v, ik, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert m.error_word(ws) == 0
        return out, sel, nsel

    def both(self):
        got, want = self.run(self.codes, ik_exp=self.exp), self.run(self.values())
        assert torch.equal(got[2], want[2])
        assert torch.equal(got[1], want[1])
        assert torch.isfinite(want[0]).all() and torch.equal(got[0], want[0])


@pytest.mark.parametrize("H,G", [(1, 16), (2, 5), (4, 16), (8, 4)])
@pytest.mark.parametrize("page", [0, 64, 256])
def test_decode_rows(H, G, page):
    Sparse([(1, 5000), (1, 1), (1, 64), (1, 65), (1, 1100), (1, 20000)], H, G, page, seed=H).both()


@pytest.mark.parametrize("H", [1, 2, 4, 8])
@pytest.mark.parametrize("ik_heads", [0, 1])
def test_drafted_windows(H, ik_heads):
    Sparse([(3, 3000), (8, 8), (2, 129), (5, 4099), (1, 700)], H, 8, 64, ik_heads, seed=H).both()


@pytest.mark.parametrize("H", [1, 4])
@pytest.mark.parametrize("page", [0, 128])
@pytest.mark.parametrize("ik_heads", [0, 1])
def test_prompt_chunks(H, page, ik_heads):
    Sparse([(300, 2000), (9, 9), (128, 128), (77, 5000), (1000, 1300)], H, 4, page, ik_heads, seed=page).both()


@pytest.mark.parametrize("kv_int8", [False, True])
def test_mixed_batches(kv_int8):
    Sparse([(1, 3000), (200, 4000), (4, 900), (1, 5), (33, 2000)], 4, 16, 64, kv_int8=kv_int8).both()


def test_long_contexts():
    Sparse([(1, 262144), (2, 100001)], 4, 16, 0).both()
    Sparse([(20, 70000)], 4, 16, 64).both()


@pytest.mark.parametrize("H,ik_heads", [(1, 0), (2, 0), (2, 1), (8, 0), (8, 1)])
def test_every_stage_is_used_again(H, ik_heads):
    """20 units of 64 positions a multiprocessor and more, for rings of up to 12."""
    Sparse([(1, 262144), (2, 100001), (8, 50000)], H, 2, 64, ik_heads=ik_heads).both()


def test_many_sequences():
    Sparse([(1 + i % 3, 3 + (i * 37) % 700) for i in range(500)], 2, 4, 64).both()


def test_powers_far_apart():
    """Scores of 2^-100 beside such of 2^90: the products are exact, so the maxima are the same."""
    Sparse([(1, 9000), (3, 700)], 2, 8, 64, exps=(-110, 100)).both()
    Sparse([(300, 3000)], 2, 8, 64, exps=(-110, 100)).both()


@pytest.mark.parametrize("rows", [1, 4, 100])
def test_keys_that_are_not_finite(rows):
    """An exponent of -128 is a NaN: the score is passed over in its block's maximum."""
    a = Sparse([(rows, 4000)], 2, 8, 64, seed=rows)
    bad = torch.rand(a.exp.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < 0.2
    keep = a.exp.clone()
    a.exp[bad] = -128
    a.codes[bad] = 0
    got = a.run(a.codes, ik_exp=a.exp)
    lowest = a.values().clone()  # the same with keys whose scores lose against all others
    m = msa()
    pb = m.Problem(a.H, a.G, a.seqs, "cuda", ik_exp=a.exp, **a.kw)
    scores = m.index_scores(pb, a.iq, a.codes)
    R, H, ld = scores.shape
    blocks = (4000 + 63) // 64
    s = torch.nan_to_num(scores[..., :4000], nan=-math.inf)
    s = torch.nn.functional.pad(s, (0, blocks * 64 - 4000), value=-math.inf).view(R, H, blocks, 64).amax(-1)
    pos = 4000 - rows + torch.arange(R, device="cuda")
    s[torch.arange(R, device="cuda"), :, pos // 64] = math.inf
    order = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :16].sort(-1).values.int()
    assert torch.equal(got[1], order)
    assert lowest.shape == a.codes.shape and keep.shape == a.exp.shape


def test_index_scores():
    """msa_index_scores against float64: |error| <= 64 2^-24 of the sum of magnitudes (fp32 sums), here integers: none."""
    a = Sparse([(3, 700), (1, 1), (40, 333)], 4, 4, 64)
    m = msa()
    pb = m.Problem(4, 4, a.seqs, "cuda", ik_exp=a.exp, **a.kw)
    s = m.index_scores(pb, a.iq, a.codes)
    table, first = a.kw["block_table"].long(), 0
    for b, (n, L) in enumerate(a.seqs):
        t = torch.arange(L, device="cuda")
        rows = table[b][t // 64] * 64 + t % 64
        want = torch.einsum("nhd,thd->nht", a.iq[first:first + n].double(), a.values()[rows].double())
        for i in range(n):
            p = L - n + i
            assert torch.equal(s[first + i, :, :p + 1].double(), want[i, :, :p + 1])
            assert torch.isinf(s[first + i, :, p + 1:]).all()
        first += n


def quantised(y):
    """Codes and exponents of y [..., 64] from the definition, in float64."""
    top = y.abs().amax(-1)
    m, e = torch.frexp(top.cpu())  # top = m 2^e, m in [1/2, 1), and 127 = (127 / 128) 2^7  (log2 of a power of two may be off)
    e = e - 7 + (m > 127 / 128).int()
    e = torch.where(top.cpu() > 0, e, torch.full_like(e, -126)).clamp(min=-126).double().to(y.device)
    return torch.round(y * torch.exp2(-e)[..., None]), e


@pytest.mark.parametrize("H,ik_heads", [(1, 0), (2, 0), (4, 0), (8, 0), (8, 1)])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("rope", [0, 32, 64])
def test_append(H, ik_heads, page, rope):
    """Without rotation the codes are those of the definition.  Rotated values are fp32 (half a step of 2^-24 for each of
    three operations and for cosine and sine, 2^-21 in all), so a code may round the other way where the quotient is
    within 127 2^-21 of a half, and the power of two be another where the maximum is as near 127 2^e."""
    m = msa()
    g = torch.Generator(device="cuda").manual_seed(H + page)
    seqs = [(1, 1), (3, 200), (70, 70), (1, 4000), (400, 1000)]
    kw = {}
    if page:
        kw["block_table"], T = paged(seqs, page)
        kw["page_size"] = page
    else:
        starts = [5, 300, 700, 1000, 6000]
        kw["cache_starts"], T = starts, 8000
    KH, R = 1 if ik_heads else H, sum(n for n, _ in seqs)
    exp = torch.full((T, KH), 77, dtype=torch.int8, device="cuda")
    codes = torch.full((T, KH, 64), 55, dtype=torch.int8, device="cuda")
    pb = m.Problem(H, 2, seqs, "cuda", cache_tokens=T, ik_heads=ik_heads, ik_exp=exp, **kw)
    k, v = (torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    new = torch.randn(R, H, 128, generator=g, device="cuda").bfloat16()
    wide = torch.randn(R, KH * 64 + 16, generator=g, device="cuda").bfloat16()
    wide *= torch.exp2(torch.randint(-30, 30, (R, 1), generator=g, device="cuda").float()).bfloat16()
    ik = wide[:, :KH * 64].view(R, KH, 64)
    ik[7] = 0
    ik[8, 0, 1:] = 0
    ik[9, 0] = 127 * 0.125  # the largest code, at a power of two
    ik[10, 0] = 127.5 * 0.125
    r = m.Rope(rope, rope, theta=1e4) if rope else None
    m.append_cache(pb, new, new, k, v, new_ik=ik, ik=codes, rope=r)
    torch.cuda.synchronize()
    rows, where = [], []
    for b, (n, L) in enumerate(seqs):
        t = torch.arange(L - n, L, device="cuda")
        rows.append(kw["block_table"][b].long()[t // page] * page + t % page if page else starts[b] + t)
        where.append(t)
    rows, where = torch.cat(rows), torch.cat(where)[None]
    y = rotate_ref(ik, rope, where) if rope else ik.double()
    want, e = quantised(y)
    got, ge = codes[rows].double(), exp[rows].double()
    if rope == 0:
        assert torch.equal(ge, e) and torch.equal(got, want)
    else:
        top = y.abs().amax(-1)
        near = (top / 127 / torch.exp2(torch.round(torch.log2(top.clamp_min(1e-300) / 127))) - 1).abs() < 2.0 ** -20
        assert ((ge == e) | near).all()
        same = (ge == e)[..., None]
        quotient = y * torch.exp2(-e)[..., None]
        half = (quotient.abs() % 1 - 0.5).abs() < 127 * 2.0 ** -20
        assert ((got == want) | half | ~same).all()
        assert (got - want).abs()[same.expand_as(got)].max() <= 1
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert (codes[others] == 55).all() and (exp[others] == 77).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("dim", [32, 64])
def test_codes_of_a_rotation_in_64_bits(interleaved, axes, dim):
    """Codes and exponents are those of the rotation in 64 bits (one in 32 bits chooses the other neighbour of about one value
    in a million; the reference's angles, 1e-11 off, of one in a thousand millions)."""
    m = msa()
    g = torch.Generator(device="cuda").manual_seed(axes)
    R, H = 1200, 4
    exp = torch.zeros(R, H, dtype=torch.int8, device="cuda")
    codes = torch.zeros(R, H, 64, dtype=torch.int8, device="cuda")
    pb = m.Problem(H, 1, [(R, R)], "cuda", ik_exp=exp)
    k, v = (torch.zeros(R, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    new = torch.randn(R, H, 128, generator=g, device="cuda").bfloat16()
    ik = torch.randn(R, H, 64, generator=g, device="cuda").bfloat16()
    where = torch.randint(1, 20000, (axes, R), generator=g, device="cuda", dtype=torch.int32)
    axis = [j % axes for j in range(dim // 2)] if axes > 1 else None
    r = m.Rope(dim, dim, theta=1e4, axes=axes, axis=axis, index_axis=axis, interleaved=interleaved)
    m.append_cache(pb, new, new, k, v, new_ik=ik, ik=codes, rope=r, positions=where)
    y = rotate_ref(ik, dim, where, interleaved=interleaved, axis=axis)
    _, e = quantised(y)
    want = torch.round(y * ((1023 - e.long()) << 52).view(torch.float64)[..., None])
    assert torch.equal(exp.double(), e)
    assert torch.equal(codes.double(), want)


def test_append_values_at_the_ends_of_the_range():
    m = msa()
    inf, nan = float("inf"), float("nan")
    heads = torch.zeros(8, 1, 64)
    heads[0, 0, :2] = torch.tensor([3.3895313892515355e38, -1.0])   # the largest bf16
    heads[1, 0, :2] = torch.tensor([1.1754943508222875e-38, 2e-39])  # the least normal one
    heads[2, 0, 5] = 9.2e-41                                         # subnormal
    heads[3, 0, 63] = inf
    heads[4, 0, 0] = nan
    heads[5, 0, 0] = -inf
    heads[6, 0] = 1.0
    exp = torch.zeros(8, 1, dtype=torch.int8, device="cuda")
    codes = torch.full((8, 1, 64), 3, dtype=torch.int8, device="cuda")
    pb = m.Problem(1, 1, [(8, 8)], "cuda", cache_tokens=8, ik_exp=exp)
    kv = torch.zeros(8, 1, 128, dtype=torch.bfloat16, device="cuda")
    new = heads.bfloat16().cuda()
    m.append_cache(pb, kv.clone(), kv.clone(), kv, kv.clone(), new_ik=new, ik=codes)
    torch.cuda.synchronize()
    assert exp[:, 0].tolist() == [122, -126, -126, -128, -128, -128, -6, -126]
    finite = torch.tensor([0, 1, 2, 6, 7], device="cuda")
    back = codes[finite].double() * torch.exp2(exp[finite].double())[..., None]
    step = torch.exp2(exp[finite].double())[..., None]
    assert ((back - new[finite].double()).abs() <= step / 2).all()
    assert (codes[3:6] == 0).all()


def test_write_and_read_together():
    """A prompt written in two chunks, then decoding steps: every step's forward chooses what a bf16 cache of the written
    values gives."""
    m = msa()
    g = torch.Generator(device="cuda").manual_seed(5)
    H, G, page, L = 2, 4, 64, 1500
    table, T = paged([(1, 2000)], page)
    exp = torch.zeros(T, H, dtype=torch.int8, device="cuda")
    codes = torch.zeros(T, H, 64, dtype=torch.int8, device="cuda")
    k, v = (torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = 0
    for n in (1000, L - 1000, 1, 1, 3, 8, 20):
        at += n
        kw = dict(block_table=table, page_size=page, cache_tokens=T)
        pb = m.Problem(H, G, [(n, at)], "cuda", ik_exp=exp, **kw)
        new = torch.randn(n, H, 128, generator=g, device="cuda").bfloat16()
        ik = torch.randint(-60, 61, (n, H, 64), generator=g, device="cuda").bfloat16()
        q = torch.randn(n, H * G, 128, generator=g, device="cuda").bfloat16()
        iq = torch.randint(-8, 9, (n, H, 64), generator=g, device="cuda").bfloat16()
        m.append_cache(pb, new, new, k, v, new_ik=ik, ik=codes)
        got = m.forward(pb, q, iq, k, v, codes)
        values = torch.ldexp(codes.float(), exp[..., None].int()).bfloat16()
        want = m.forward(m.Problem(H, G, [(n, at)], "cuda", **kw), q, iq, k, v, values)
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_a_captured_forward_is_replayed():
    m = msa()
    a = Sparse([(1, 3000), (4, 2000)], 4, 16, 64)
    pb = m.Problem(a.H, a.G, a.seqs, "cuda", ik_exp=a.exp, **a.kw)
    ws, out, (sel, nsel) = pb.workspace(), pb.new_out(), pb.new_sel()
    want = [x.clone() for x in m.forward(pb, a.q, a.iq, a.k, a.v, a.codes, workspace=ws)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(pb, a.q, a.iq, a.k, a.v, a.codes, out=out, sel=sel, nsel=nsel, workspace=ws)
    for _ in range(3):
        out.zero_(), sel.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(sel, want[1]) and torch.equal(nsel, want[2])


def test_a_bad_page_is_reported():
    m = msa()
    for n in (1, 40):
        a = Sparse([(n, 700)], 2, 4, 64)
        a.kw["block_table"][0, 3] = 1 << 20
        pb = m.Problem(a.H, a.G, a.seqs, "cuda", ik_exp=a.exp, **a.kw)
        ws = pb.workspace()
        m.forward(pb, a.q, a.iq, a.k, a.v, a.codes, workspace=ws)
        torch.cuda.synchronize()
        assert m.error_word(ws) == m.ERR_BAD_METADATA
