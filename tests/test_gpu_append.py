"""msa_append_cache against a plain 64-bit implementation.

Bounds.  The phase x turns / 2^64 is exact modulo a turn up to the rounding of
the tables (2^-52 of the angle); its upper 32 bits become an fp32 number of
half turns (2^-25) and sincospi adds at most 2 units of 2^-24, so cos and sin
are within 2^-22.  The rotation's products and sum in fp32 add 3 2^-24.  A
rotated value is thus within 2^-21 (|x_a| + |x_b|) of the formula's, plus half
a step of bf16 where it is rounded to that.  A code is within half a step of
the rotated value over the scale, which is within 2^-21 relative (two more
fp32 roundings) of max |y| / 127."""
import math

import pytest
import torch

from dense_common import half_step, rotate_ref
from gpu_common import msa

pytestmark = pytest.mark.gpu

H_STEP = half_step(torch.bfloat16)


class New:
    def __init__(self, seqs, H, G, int8=False, page=0, seed=0, shared=False, far=False, spare=0):
        m = msa()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.seqs, self.H, self.G, self.int8 = seqs, H, G, int8
        self.KH = 1 if shared else H
        R = sum(n for n, _ in seqs)
        self.R, RR = R, R + spare
        widths = [H * G * 128, H * 128, H * 128, H * 64, self.KH * 64]
        # one projection's output, its parts at odd multiples of 8 elements, padded rows
        wide = torch.randn(RR, sum(widths) + 8 + 24, generator=g, device="cuda").bfloat16()
        parts = torch.split(wide[:, 8:8 + sum(widths)], widths, dim=1)
        self.q, self.k, self.v, self.iq, self.ik = (
            p.view(RR, -1, d) for p, d in zip(parts, (128, 128, 128, 64, 64)))
        B = len(seqs)
        self.table = self.starts = None
        kw = {"ik_heads": 1 if shared else 0}
        if page:
            need = [-(-L // page) for _, L in seqs]
            ids = torch.randperm(sum(need) + 1, generator=torch.Generator().manual_seed(seed)).tolist()
            t = [[-1] * max(need) for _ in range(B)]
            at = 0
            for b, c in enumerate(need):
                t[b][:c] = ids[at:at + c]
                at += c
            self.table, T = torch.tensor(t, dtype=torch.int32, device="cuda"), (sum(need) + 1) * page
            kw.update(block_table=self.table, page_size=page)
        else:
            self.starts, at = [], 2
            for _, L in seqs:
                self.starts.append(at)
                at += L + 1
            T = at
            kw.update(cache_starts=self.starts)
        self.T, self.page = T, page
        held = torch.int8 if int8 else torch.bfloat16
        self.kc, self.vc = (torch.full((T, H, 128), 77, dtype=held, device="cuda") for _ in range(2))
        self.ikc = torch.full((T, self.KH, 64), 77, dtype=torch.bfloat16, device="cuda")
        if int8:
            self.ks, self.vs = (torch.full((T, H), 77.0, device="cuda") for _ in range(2))
            kw.update(k_scale=self.ks, v_scale=self.vs)
        self.pb = m.Problem(H, G, seqs, "cuda", cache_tokens=T, **kw)
        self.pb.total_rows = self.pb.c.total_rows = RR
        rows, pos = [], []
        for b, (n, L) in enumerate(seqs):
            t = torch.arange(L - n, L, device="cuda")
            pos.append(t)
            rows.append(self.table[b].long()[t // page] * page + t % page if page else self.starts[b] + t)
        self.rows, self.pos = torch.cat(rows), torch.cat(pos)

    def run(self, rope=None, positions=None, ws=None, **kw):
        m = msa()
        ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        got = m.append_cache(self.pb, self.k, self.v, self.kc, self.vc, new_ik=self.ik, ik=self.ikc, q=self.q,
                             iq=self.iq, rope=rope, positions=positions, workspace=ws, **kw)
        torch.cuda.synchronize()
        assert m.error_word(ws) == 0
        return got

    def check(self, q, iq, dim=0, idim=0, where=None, **kw):
        R = self.R
        where = self.pos[None] if where is None else where[:, :R]
        axis, iaxis = kw.pop("axis", None), kw.pop("index_axis", None)

        def near(got, x, d, ax, name):
            x = x[:R].double()
            y = rotate_ref(x, d, where, axis=ax, **kw)
            z = rotate_ref(x.abs(), d, torch.zeros_like(where), axis=ax, **kw)  # |x_a| of each, then its partner's
            j = torch.arange(d // 2)
            a, b = (2 * j, 2 * j + 1) if kw.get("interleaved") else (j, j + d // 2)
            both = z.clone()
            both[..., a], both[..., b] = z[..., a] + z[..., b], z[..., a] + z[..., b]
            bound = both * 2.0 ** -21 + y.abs() * H_STEP
            if d == 0:
                assert torch.equal(got.double(), y), name
            assert ((got.double() - y).abs() <= bound).all(), name
            assert torch.equal(got[..., d:], x[..., d:].bfloat16()), name
            return y, both

        near(q[:R], self.q, dim, axis, "q")
        near(iq[:R], self.iq, idim, iaxis, "iq")
        near(self.ikc[self.rows], self.ik, idim, iaxis, "ik")
        for name, x, cache, d in (("k", self.k, self.kc, dim), ("v", self.v, self.vc, 0)):
            if not self.int8:
                near(cache[self.rows], x, d, axis if d else None, name)
                continue
            scale = (self.ks if name == "k" else self.vs)[self.rows]
            code = cache[self.rows].double()
            x = x[:R].double()
            y = rotate_ref(x, d, where, axis=axis if d else None, **kw)
            top = y.abs().amax(-1)
            slack = 2.0 ** -21 * x.abs().amax(-1) * 2
            assert ((scale.double() - top / 127).abs() <= slack / 127 + 2.0 ** -22 * top / 127).all(), name
            assert ((code * scale.double()[..., None] - y).abs() <=
                    (0.5 + 2.0 ** -14) * scale.double()[..., None] + slack[..., None]).all(), name
        rest = torch.ones(self.T, dtype=torch.bool, device="cuda")
        rest[self.rows] = False
        for c in (self.kc, self.vc, self.ikc) + ((self.ks, self.vs) if self.int8 else ()):
            assert (c[rest] == 77).all(), "a cache row of another position was written"


SEQS = [(1, 1), (1, 64), (1, 65), (7, 130), (64, 64), (65, 200), (3, 4000)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("page", [0, 64, 256])
@pytest.mark.parametrize("H,G", [(1, 1), (4, 16), (8, 3)])
def test_rotated_and_stored(H, G, page, int8):
    m = msa()
    for dim, idim, inter in ((0, 0, False), (64, 64, False), (128, 32, True), (16, 16, False), (96, 48, False)):
        x = New(SEQS, H, G, int8, page, seed=dim)
        q, iq = x.run(m.Rope(dim, idim, interleaved=inter) if dim else None)
        x.check(q, iq, dim, idim, interleaved=inter)


@pytest.mark.parametrize("int8", [False, True])
def test_several_axes_and_any_positions(int8):
    m = msa()
    x = New([(300, 300), (5, 17)], 2, 4, int8)
    pos = torch.randint(-(1 << 21), 1 << 21, (3, 305), device="cuda", dtype=torch.int32)
    axis = torch.tensor([0, 1, 2, 2, 1, 0, 0, 0] * 4)
    rope = m.Rope(64, 32, theta=5e6, axes=3, axis=axis, index_axis=axis[:16])
    q, iq = x.run(rope, pos)
    x.check(q, iq, 64, 32, pos, theta=5e6, axis=axis.tolist(), index_axis=axis[:16].tolist())


def test_far_positions_keep_their_angles():
    m = msa()
    x = New([(2, (1 << 21)), (1, 100001)], 1, 2, page=1 << 20)
    q, iq = x.run(m.Rope(128, 64))
    x.check(q, iq, 128, 64)


def test_shared_index_key_and_rows_behind_the_last_sequence():
    m = msa()
    x = New([(1, 9), (12, 30)], 4, 2, shared=True, spare=3)
    q, iq = x.run(m.Rope(32, 32))
    x.check(q, iq, 32, 32)


def test_without_rotation_the_codes_are_the_formulas():
    x = New([(200, 200)], 2, 1, int8=True)
    x.v[3, 0] = 0
    x.v[4, 1] = x.v[4, 1].abs().clamp(max=1e-38) * 2.0 ** -10  # subnormal scales
    x.run()
    for new, cache, scale in ((x.k, x.kc, x.ks), (x.v, x.vc, x.vs)):
        y = new.float().cpu()
        s = y.abs().amax(-1) / 127
        code = torch.where(s[..., None] > 0, y / s[..., None], torch.zeros(())).round().clamp(-127, 127)
        assert torch.equal(scale[x.rows].cpu(), s)
        assert torch.equal(cache[x.rows].cpu().float(), code)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_heads_read_back_as_nan(bad):
    x = New([(4, 4)], 2, 1, int8=True)
    x.k[1, 1, 77] = bad
    x.run()
    row = x.rows[1]
    assert not torch.isfinite(x.ks[row, 1])
    assert (x.kc[row, 1] == 0).all()
    assert torch.isnan(x.kc[row, 1].float() * x.ks[row, 1]).all()
    assert torch.isfinite(x.ks[row, 0]) and torch.isfinite(x.ks[x.rows[0]]).all()


def test_parts_may_be_left_out_and_queries_rotated_in_place():
    m = msa()
    x = New([(5, 50)], 2, 3)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    q, iq = m.append_cache(x.pb, x.k, x.v, x.kc, x.vc, rope=m.Rope(64), workspace=ws)
    assert q is None and iq is None
    torch.cuda.synchronize()
    y = rotate_ref(x.k, 64, x.pos[None])
    assert ((x.kc[x.rows].double() - y).abs() <= 2.0 ** -20 * 8 + y.abs() * H_STEP).all()
    assert (x.ikc == 77).all()


@pytest.mark.parametrize("int8", [False, True])
def test_bad_metadata_is_reported_and_not_stored(int8):
    m = msa()
    x = New([(3, 100), (2, 70)], 2, 2, int8, page=64)
    x.pb.block_table[0, 1] = 1000
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    m.append_cache(x.pb, x.k, x.v, x.kc, x.vc, workspace=ws)
    torch.cuda.synchronize()
    assert m.error_word(ws) == m.ERR_BAD_METADATA
    assert (x.kc[x.rows[3:]] != 77).any()
    rest = torch.ones(x.T, dtype=torch.bool, device="cuda")
    rest[x.rows[3:]] = False
    assert (x.kc[rest] == 77).all()


def test_a_run_of_writer_and_both_attentions():
    """A prompt and then single tokens: written by append_cache, read by the
    sparse and the dense attention, eagerly and from a captured step."""
    from dense_common import dense_ref
    m = msa()
    H, G, page, steps, first = 2, 8, 64, 5, 130
    g = torch.Generator(device="cuda").manual_seed(1)
    T = 8 * page
    table = torch.tensor([[5, 1, 7, 2]], dtype=torch.int32)
    kc, vc = (torch.full((T, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ikc = torch.zeros(T, H, 64, dtype=torch.bfloat16, device="cuda")
    rope = m.Rope(64, 32, theta=1e6)
    done = 0
    for step in range(steps + 1):
        n = first if step == 0 else 1
        L = done + n
        pb = m.Problem(H, G, [(n, L)], "cuda", block_table=table, page_size=page, cache_tokens=T)
        new = {x: torch.randn(n, h, d, generator=g, device="cuda").bfloat16()
               for x, h, d in (("q", H * G, 128), ("k", H, 128), ("v", H, 128), ("iq", H, 64), ("ik", H, 64))}
        wa, wd, wf = (torch.full((s,), 255, dtype=torch.uint8, device="cuda")
                      for s in (256, pb.dense_workspace_size(), pb.workspace_size()))

        def one():
            q, iq = m.append_cache(pb, new["k"], new["v"], kc, vc, new_ik=new["ik"], ik=ikc, q=new["q"], iq=new["iq"],
                                   rope=rope, workspace=wa)
            dense = m.dense_forward(pb, q, kc, vc, workspace=wd)
            # the sparse kernels multiply the rest of a kept block by zero weights, so it has to be finite for them
            sparse, _, _ = m.forward(pb, q, iq, kc.nan_to_num(), vc.nan_to_num(), ikc, workspace=wf)
            return q, dense, sparse

        if step == steps:  # the same step captured, its result replayed
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                q, dense, sparse = one()
            graph.replay()
        else:
            q, dense, sparse = one()
        torch.cuda.synchronize()
        assert m.error_word(wa) == 0 and m.error_word(wd) == 0 and m.error_word(wf) == 0
        t = table[0].cuda()
        ref, bound = dense_ref([(n, L)], H, G, q, kc, vc, 1 / math.sqrt(128),
                               lambda b, p: t.long()[p // page] * page + p % page, torch.float32, 24)
        assert ((dense.double() - ref).abs() <= bound).all()
        assert (sparse.double() - ref).abs().max() <= 2e-3  # fewer blocks than top_k: every block is kept
        done = L


def test_wrong_arguments_are_refused():
    m = msa()
    x = New([(4, 9)], 2, 2)
    with pytest.raises(ValueError):
        m.append_cache(x.pb, x.k, x.v, x.kc, x.vc, new_ik=x.ik)
    with pytest.raises(ValueError):
        m.append_cache(x.pb, x.k[:3], x.v, x.kc, x.vc)
    with pytest.raises(ValueError):
        m.append_cache(x.pb, x.k.transpose(1, 2).contiguous().transpose(1, 2), x.v, x.kc, x.vc)
    with pytest.raises(TypeError):
        m.append_cache(x.pb, x.k.float(), x.v, x.kc, x.vc)
    with pytest.raises(ValueError):
        m.append_cache(x.pb, x.k, x.v, x.kc, x.vc, positions=torch.zeros(1, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        m.append_cache(x.pb, x.k, x.v, x.kc, x.vc, rope=m.Rope(32), positions=torch.zeros(2, 4, dtype=torch.int32,
                                                                                         device="cuda"))
    with pytest.raises(m.MsaError):
        m.append_cache(x.pb, x.k, x.v, x.kc, x.vc, rope=m.Rope(24))
    with pytest.raises(m.MsaError):
        m.append_cache(x.pb, x.k, x.v, x.kc, x.vc, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    odd = torch.randn(4, 2 * 128 + 4, device="cuda").bfloat16()[:, :256].view(4, 2, 128)
    with pytest.raises(m.MsaError):
        m.append_cache(x.pb, odd, x.v, x.kc, x.vc)
