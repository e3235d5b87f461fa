"""Plain 64-bit forms of the cache writer and the dense attention, and the
error bounds that their tests use, derived from the roundings the kernels
make.

Dense attention, out = sum_t w_t v_t with w = softmax(x), x_t = scale q.k_t.
  - x_t comes from 128 products of bf16 (exact in fp32) summed in fp32 in some
    order and multiplied by the scale and log2(e): |dx_t| <= (128 + 4) 2^-24 A,
    A = max_t scale sum_d |q_d k_td| (4: the scale, its product with log2(e),
    the multiply and the subtraction of the maximum, whose own error of the
    same size is common to all t and cancels in the ratio, but is counted
    again below).  An int8 key's scale is one more rounding.  A weight is off
    by a factor exp(+-2 |dx|), and its exponential by 2^-22.
  - the sums over L keys are in fp32: L 2^-24, in the numerator and in the
    denominator.
  - a weight entering the product with v is rounded to one bf16 (2^-8), two
    (2^-16) or three (2^-24) parts; int8 caches multiply it by the value's
    scale first (one more fp32 rounding, inside the L 2^-24).  f16 forms of an
    int8 cache: a weight is off by 2^-12, and in prompts with bf16 outputs keys
    and values by up to 2^-12 of themselves.  Weight and value are inside the
    2^-8 counted for one bf16 part.  The key's share, 2^-12 A of a score if all
    128 errors had one sign, is not counted: the tests hold these outputs to
    the tighter bound.
  - the output is rounded to its type: half a step, eps / 2 of its magnitude.
All but the last scale with sum_t w_t |v_t|."""
import math

import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def cache_rows(b, t, starts=None, table=None, page=0):
    """Cache rows of positions t of sequence b."""
    if table is not None:
        return table[b].long()[t // page] * page + t % page
    return starts[b] + t


def dense_ref(seqs, H, G, q, k, v, scale, rows_of, out_dtype, weight_bits, k_scale=None, v_scale=None):
    """(out, bound) in float64 on the inputs' device; weight_bits: rounding of the weights, 8, 16 or 24."""
    R, D = q.shape[0], q.shape[2]
    out = torch.full((R, H * G, D), float("nan"), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    first = 0
    for b, (n, L) in enumerate(seqs):
        if n == 0:
            continue
        rows = rows_of(b, torch.arange(L, device=q.device))
        p = torch.arange(L - n, L, device=q.device)
        for h in range(H):
            kk, vv = k[rows, h].double(), v[rows, h].double()
            if k_scale is not None:
                kk = kk * k_scale[rows, h].double()[:, None]
                vv = vv * v_scale[rows, h].double()[:, None]
            qq = q[first:first + n, h * G:(h + 1) * G].double()  # [n, G, D]
            x = scale * torch.einsum("ngd,td->ngt", qq, kk)
            hide = torch.arange(L, device=q.device)[None] > p[:, None]
            x = x.masked_fill(hide[:, None], -math.inf)
            w = torch.softmax(x, -1)
            o = torch.einsum("ngt,td->ngd", w, vv)
            wv = torch.einsum("ngt,td->ngd", w, vv.abs())
            A = (scale * torch.einsum("ngd,td->ngt", qq.abs(), kk.abs())).masked_fill(hide[:, None], 0).amax(-1)
            rel = 2 * (128 + 5) * 2.0 ** -24 * A + 2.0 ** -22 + 2 * L * 2.0 ** -24 + 2.0 ** -weight_bits
            out[first:first + n, h * G:(h + 1) * G] = o
            bound[first:first + n, h * G:(h + 1) * G] = wv * rel[..., None] + o.abs() * half_step(out_dtype)
        first += n
    return out, bound


def rotate_ref(x, dim, where, theta=10000.0, interleaved=False, axis=None):
    """x [R, heads, D] rotated in float64; where [axes, R] positions."""
    y = x.double().clone()
    for j in range(dim // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + dim // 2)
        angle = (where[axis[j] if axis is not None else 0].double() * theta ** (-2.0 * j / dim))[:, None]
        xa, xb = x[..., a].double(), x[..., b].double()
        y[..., a] = xa * angle.cos() - xb * angle.sin()
        y[..., b] = xb * angle.cos() + xa * angle.sin()
    return y
