"""The bits that msa_dense_forward's weights and keys keep, form by form.

A rounding is off by half a step at most: 2^-8 for one bf16 part of a weight,
2^-16 for two, 2^-11 for one f16 part.  Values of both signs make the outputs
small beside sum_t w_t |v_t|, which the weights' rounding scales with, so that
the rounding of the outputs hides none of it."""
import math

import pytest
import torch

from dense_common import dense_ref, half_step
from test_gpu_dense import Batch

pytestmark = pytest.mark.gpu


def balanced(seqs, H, G, int8, page=64, seed=1):
    b = Batch(seqs, H, G, int8, page, torch.bfloat16, seed=seed, q_gain=1.0)
    if not int8:
        b.v = torch.randn(b.v.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()
    return b


def reference(b, bits):
    return dense_ref(b.seqs, b.H, b.G, b.q, b.k, b.v, float(torch.tensor(b.scale)), b.rows_of, torch.bfloat16, bits,
                     b.k_scale, b.v_scale)


def with_fewer_bits(b, weight_type):
    """The formula with each weight, over the row's largest, rounded to weight_type, in 64 bits otherwise."""
    out, first = [], 0
    for i, (n, L) in enumerate(b.seqs):
        rows = b.rows_of(i, torch.arange(L, device="cuda"))
        k, v = b.k[rows].double(), b.v[rows].double()
        if b.int8:
            k, v = k * b.k_scale[rows].double()[..., None], v * b.v_scale[rows].double()[..., None]
        q = b.q[first:first + n].double().view(n, b.H, b.G, 128)
        x = b.scale * torch.einsum("nhgd,thd->nhgt", q, k)
        hide = torch.arange(L, device="cuda")[None] > torch.arange(L - n, L, device="cuda")[:, None]
        x = x.masked_fill(hide[:, None, None], -math.inf)
        w = (x - x.amax(-1, keepdim=True)).exp()
        o = torch.einsum("nhgt,thd->nhgd", w.to(weight_type).double(), v) / w.sum(-1)[..., None]
        out.append(o.reshape(n, b.H * b.G, 128))
        first += n
    return torch.cat(out).bfloat16()


@pytest.mark.parametrize("seqs,G", [([(1, L) for L in (3, 64, 100, 257, 1000)], 16), ([(1, 300), (1, 77)], 5),
                                    ([(4, 130), (2, 90), (4, 4)], 4), ([(8, 200), (3, 64)], 2)])
def test_decode_rows_and_small_windows_keep_two_parts(seqs, G):
    b = balanced(seqs, 2, G, False)
    ref, bound = reference(b, 16)
    got = b.run()
    assert ((got.double() - ref).abs() <= bound).all()
    one = with_fewer_bits(b, torch.bfloat16)
    assert ((one.double() - ref).abs() > bound).any()  # (the bound would tell one part)


@pytest.mark.parametrize("seqs,G", [([(1, L) for L in (3, 64, 100, 257, 1000)], 16), ([(4, 130), (2, 90), (8, 8)], 16),
                                    ([(8, 200), (3, 64)], 2)])
def test_int8_decode_rows_and_windows_keep_11_bits(seqs, G):
    b = balanced(seqs, 2, G, True)
    ref, bound = reference(b, 11)
    got = b.run()
    assert ((got.double() - ref).abs() <= bound).all()
    fewer = with_fewer_bits(b, torch.bfloat16)
    assert ((fewer.double() - ref).abs() > bound).any()


@pytest.mark.parametrize("n,L", [(20, 300), (100, 1000), (33, 33)])
@pytest.mark.parametrize("large", [16, 64])
def test_int8_prompts_with_one_large_key_channel(n, L, large):
    """The f16 copy's keys are off by 2^-11 of themselves each: a score by up to 2^-11 of sum_d |q_d k_d|, which a large
    channel makes large beside the scores' spread.  Beside it the weights' one part (f16, 2^-11), and the values' 2^-11."""
    b = balanced([(n, L)], 2, 16, True)
    g = torch.Generator(device="cuda").manual_seed(3)
    b.k.copy_(torch.randint(-127 // large, 127 // large + 1, b.k.shape, generator=g, device="cuda", dtype=torch.int8))
    b.k[..., 7] = torch.randint(100, 128, b.k.shape[:2], generator=g, device="cuda", dtype=torch.int8)
    b.pb.k_scale.mul_(large / 4)
    b.k_scale = b.pb.k_scale
    ref, bound = reference(b, 10)  # (2^-11 twice)
    _, without = reference(b, 60)
    rows = b.rows_of(0, torch.arange(L, device="cuda"))
    k = b.k[rows].double() * b.k_scale[rows].double()[..., None]
    A = b.scale * torch.einsum("nhgd,thd->nhgt", b.q.double().view(n, 2, 16, 128).abs(), k.abs()).amax(-1).reshape(n, 32)
    # sum_t w_t |v_t|, from the bound's share of the weights
    wv = (bound - without) / (2.0 ** -10 - 2.0 ** -60)
    got = b.run()
    assert ((got.double() - ref).abs() <= bound + 2 * 2.0 ** -11 * A[..., None] * wv).all()
    # at random rather than worst: in the 2-norm the keys' share stays below the outputs' own rounding, half a step
    assert (got.double() - ref).norm() <= 2 * half_step(torch.bfloat16) * ref.norm()
