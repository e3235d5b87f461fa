"""msa_dense_forward on caches whose scales, keys or lengths strain its number
formats."""
import pytest
import torch

from gpu_common import msa
from test_gpu_dense import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,L", [(9, 9), (40, 60), (200, 300)])
@pytest.mark.parametrize("value,rest", [(2.0 ** 40, 1.0), (1.0, 2.0 ** -40), (2.0 ** 20, 1.0), (2.0 ** 24, 1.0), (2.0 ** 30, 1.0)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_int8_prompts_behind_which_a_far_larger_value_lies(n, L, value, rest, out):
    """The last token's value scale leaves those of the tokens before it, in the same block, far behind."""
    b = Batch([(n, L), (n, L)], 2, 16, True, 0, out, seed=n)
    rows = b.rows_of(0, torch.arange(L, device="cuda"))
    b.pb.v_scale[rows] *= rest
    b.pb.v_scale[rows[-1]] *= value / rest
    b.check()


@pytest.mark.parametrize("n,L", [(9, 9), (40, 60), (200, 300)])
@pytest.mark.parametrize("key,rest", [(2.0 ** 60, 1.0), (2.0 ** 24, 1.0), (1.0, 2.0 ** -50)])
def test_int8_prompts_behind_which_a_far_larger_key_lies(n, L, key, rest):
    """The same of the keys; the rows that do not see it must not tell.  (In the last row the large key's score is
    far above or below all others, and rounding decides nothing.)"""
    b = Batch([(n, L), (n, L)], 2, 16, True, 0, torch.bfloat16, seed=n)
    if rest != 1:  # tiny keys whose scores matter: queries that are large in turn
        b.q[:n] *= 2.0 ** 50
    rows = b.rows_of(0, torch.arange(L, device="cuda"))
    b.pb.k_scale[rows] *= rest
    b.pb.k_scale[rows[-1]] *= key / rest
    ref, bound = b.ref()
    got = b.run()
    keep = torch.ones(2 * n, dtype=torch.bool, device="cuda")
    keep[n - 1] = False
    assert torch.isfinite(got).all()
    assert ((got.double() - ref).abs() <= bound)[keep].all()


@pytest.mark.parametrize("n", [2, 3, 8])
@pytest.mark.parametrize("L", [8, 64, 66, 300])
@pytest.mark.parametrize("G", [2, 16])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_int8_windows_whose_later_values_are_far_larger(n, L, G, out):
    for later in (2.0 ** 20, 2.0 ** 40, 2.0 ** 90, 2.0 ** -40):
        b = Batch([(n, L), (n, L)], 4, G, True, 0, out, seed=n)
        rows = b.rows_of(0, torch.arange(L, device="cuda"))
        b.pb.v_scale[rows[L - n + 1:]] *= later
        b.check()
        b.pb.v_scale[rows[:L - n + 1]] = 0  # nothing but the later ones
        b.check()


@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("first", [32, 70, 128])
def test_scores_of_minus_infinity_weigh_nothing(first, out, n):
    """Keys with an infinity against a negative query, from the first position on; a chunk's last value is NaN, so
    that rows before it are computed again.  The other weights sum to 1 and are off by 2^-8 of themselves at most, the
    output by half a step of bf16, 2^-8 of itself: with the fp32 sums (below 2^-10) less than 2.5 2^-8 max |v|."""
    b = Batch([(n, 300)], 2, 16, False, 0, out, seed=first)
    rows = b.rows_of(0, torch.arange(300, device="cuda"))
    b.q[..., 5] = -1 - b.q[..., 5].abs()
    b.k[rows[:first], :, 5] = float("inf")
    ref, _ = b.ref()
    most = b.v[rows].abs().max().double()
    live = n
    if n > 8:
        b.v[rows[-1]] = float("nan")
        live = n - 1
    got = b.run()
    assert ((got.double() - ref).abs() <= 2.5 * 2.0 ** -8 * most)[:live].all()


C = 1 + 2.0 ** -7  # a value whose sums need every bit


def long_batch(B, n, G, int8, length=1 << 21, H=8, seed=1):
    """B sequences that share one cache of `length` positions; every value is C."""
    m = msa()
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = {}
    if int8:
        k = torch.randint(-127, 128, (length, H, 128), generator=g, device="cuda", dtype=torch.int8)
        v = torch.full((length, H, 128), 1, device="cuda", dtype=torch.int8)
        kw = {"k_scale": torch.full((length, H), 1 / 64, device="cuda"), "v_scale": torch.full((length, H), C, device="cuda")}
    else:
        k = torch.randn(length, H, 128, generator=g, device="cuda", dtype=torch.bfloat16)
        v = torch.full((length, H, 128), C, device="cuda", dtype=torch.bfloat16)
    pb = m.Problem(H, G, [(n, length)] * B, "cuda", out_dtype=torch.bfloat16, cache_tokens=length, cache_starts=[0] * B, **kw)
    q = torch.randn(B * n, H * G, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    return m, pb, q, k, v


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B,n,G", [(160, 1, 4), (19, 4, 16), (1, 304, 16)])
def test_the_longest_contexts_do_not_drift(B, n, G, int8):
    """Every value is C, so every output is, whatever the weights are.  A CTA walks all 2^21 positions.  Rounded
    weights differ from the summed ones at random (2^-8 L^-1/2 of the sum) and the sums of 32 bits are off by less
    than 2^-10, together below half a step of bf16 (2^-8), so the output is C itself; sums that lose something in the
    same direction 10^5 times are not."""
    m, pb, q, k, v = long_batch(B, n, G, int8)
    ws = pb.dense_workspace()
    out = m.dense_forward(pb, q, k, v, workspace=ws)
    torch.cuda.synchronize()
    assert m.error_word(ws) == 0
    assert (out.float() == C).all(), (out.float().min().item(), out.float().max().item())


@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_int8_values_that_are_all_zero(n, out):
    """Scales of zero everywhere, and everywhere but in the last, or the first, few positions."""
    for keep in (slice(0, 0), slice(295, 300), slice(0, 3)):
        b = Batch([(n, 300), (n, 200)], 2, 16, True, 64, out, seed=n)
        rows = b.rows_of(0, torch.arange(300, device="cuda"))
        kept = b.pb.v_scale[rows[keep]].clone()
        b.pb.v_scale[rows] = 0
        b.pb.v_scale[rows[keep]] = kept
        b.check()
        if keep.stop == 0:
            assert (b.run()[:n] == 0).all()
