"""msa_append_cache, index keys of 8 bits: the codes and exponents of heads
whose rotated values lie so near to a half, to where the exponent changes or
past 32 bits' range that a rotation in 32 bits decides otherwise.  The values
are searched for in float64, at least 2e-9 of the border away: the reference's
own angles are good to 1e-11."""
import pytest
import torch

from dense_common import rotate_ref
from gpu_common import msa
from test_gpu_index8 import quantised

pytestmark = pytest.mark.gpu


def _pairs(where):
    """All bf16 pairs (a, b) of 2^-9 to 2 in size with a positive; a cos - b sin and b cos + a sin of them in float64, and
    the first of the two in float32."""
    sizes = torch.cat([(1 + torch.arange(128, device="cuda", dtype=torch.float64) / 128) * 2.0 ** e for e in range(-9, 1)])
    a, b = torch.meshgrid(sizes, torch.cat([sizes, -sizes]), indexing="ij")
    t = torch.tensor(float(where), dtype=torch.float64, device="cuda")
    y32 = a.float() * t.cos().float() - b.float() * t.sin().float()
    return a, b, a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin(), y32.double()


def near_a_half(where):
    """Pairs whose first rotated value lies next to a half of the step 2^-6 (both are below 1.9, so that this stays the
    step), on the other side of it in float32."""
    a, b, y, z, y32 = _pairs(where)
    d = ((y * 64).abs() % 1 - 0.5).abs()
    ok = (d > 2e-9) & (y.abs() < 1.9) & (z.abs() < 1.9) & (torch.round(y32 * 64) != torch.round(y * 64))
    return torch.stack([a[ok], b[ok]], 1)


def near_the_largest(where):
    """Pairs whose first rotated value, the larger one, lies next to 127 2^-6, on the other side of it in float32."""
    a, b, y, z, y32 = _pairs(where)
    ok = ((y.abs() * 64 / 127 - 1).abs() > 2e-9) & (z.abs() < y.abs()) & ((y32.abs() * 64 > 127) != (y.abs() * 64 > 127))
    return torch.stack([a[ok], b[ok]], 1)


def search(kind):
    """Four positions that have such pairs, and the pairs."""
    found = []
    for p in torch.randint(1, 30000, (2000,), generator=torch.Generator().manual_seed(11)).tolist():
        pairs = kind(p)
        if len(pairs) > 0:
            found.append((p, pairs))
        if len(found) == 4:
            return found
    raise AssertionError("too few cases")


def write(ik, where, interleaved, dim=32):
    m = msa()
    R, H, _ = ik.shape
    exp = torch.full((R, H), 77, dtype=torch.int8, device="cuda")
    codes = torch.full((R, H, 64), 55, dtype=torch.int8, device="cuda")
    pb = m.Problem(H, 1, [(R, R)], "cuda", ik_exp=exp)
    k, v = (torch.zeros(R, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    new = torch.zeros(R, H, 128, dtype=torch.bfloat16, device="cuda")
    m.append_cache(pb, new, new, k, v, new_ik=ik, ik=codes, rope=m.Rope(dim, dim, theta=1e4, interleaved=interleaved),
                   positions=where)
    torch.cuda.synchronize()
    return codes, exp


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", [near_a_half, near_the_largest])
@pytest.mark.parametrize("H,R", [(1, 300), (4, 40), (8, 7400)])
def test_values_next_to_a_border(H, R, kind, interleaved):
    """Every head of every row is such a head (8 heads and 7,400 rows: sixteen rows a CTA, all of which it rotates again)."""
    found = search(kind)
    partner = 1 if interleaved else 16
    ik = torch.zeros(R, H, 64, dtype=torch.bfloat16, device="cuda")
    if kind is near_a_half:
        ik[..., 40] = 1.0  # past the rotated ones: the largest, so that the step is 2^-6
    where = torch.tensor([found[r % 4][0] for r in range(R)], dtype=torch.int32, device="cuda")[None]
    for i, (_, pairs) in enumerate(found):
        rows = torch.arange(i, R, 4, device="cuda")
        pick = (torch.arange(len(rows), device="cuda")[:, None] * H + torch.arange(H, device="cuda")) % len(pairs)
        ik[rows, :, 0] = pairs[pick, 0].bfloat16()
        ik[rows, :, partner] = pairs[pick, 1].bfloat16()
    codes, exp = write(ik, where, interleaved)
    y = rotate_ref(ik, 32, where, interleaved=interleaved)
    _, e = quantised(y)
    step = ((1023 + e.long()) << 52).view(torch.float64)[..., None]
    assert torch.equal(exp.double(), e)
    assert torch.equal(codes.double(), torch.round(y / step))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [4, 300, 2000])
def test_values_that_are_turned_past_32_bits(R, interleaved):
    """Two finite values near 3.4e38 turned to one of up to 4.8e38: the definition's exponent, 122.  A head that does hold a
    NaN or an infinity, among its rotated dimensions or the others, gets -128 and codes of 0."""
    H, partner = 2, 1 if interleaved else 16
    where = (torch.arange(R, device="cuda", dtype=torch.int32) % 997)[None]
    g = torch.Generator(device="cuda").manual_seed(R)
    ik = torch.randn(R, H, 64, generator=g, device="cuda").bfloat16()
    angle = where[0].double()
    size = 3.3e38
    ik[:, 0, 0] = (size * torch.sign(angle.cos())).bfloat16()
    ik[:, 0, partner] = (-size * torch.sign(angle.sin())).bfloat16()
    bad = torch.arange(R, device="cuda") % 4 == 3
    ik[bad, 1, 5] = float("inf")
    ik[1::4, 1, 60] = float("nan")
    ik[2::4, 1, 63] = -float("inf")
    codes, exp = write(ik, where, interleaved)
    y = rotate_ref(ik, 32, where, interleaved=interleaved)
    _, e = quantised(y[:, 0])
    assert (y[:, 0, 0].abs() > 3.41e38).any() and (e >= 121).all()
    assert torch.equal(exp[:, 0].double(), e)
    assert torch.equal(codes[:, 0].double(), torch.round(y[:, 0] / ((1023 + e.long()) << 52).view(torch.float64)[..., None]))
    for i in (1, 2, 3):
        assert (exp[i::4, 1] == -128).all() and (codes[i::4, 1] == 0).all()
    assert (exp[0::4, 1] > -20).all()
