// Attention over every cached position, the plain way: a thread keeps one
// (query row, query head) with its query and its running output in registers
// and walks the keys, which its CTA stages through shared memory.
//   s_t = scale q . k_t,   out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  m = max_t s_t
// in one pass with a running maximum; everything in fp32.
#include "common.cuh"
#include "internal.h"

namespace msa {

constexpr int kDsThreads = 128;
constexpr int kDsKeys = 32;

// Reads element i of a row of 8 cached values as fp32.
__device__ __forceinline__ void ds_load8(const void* base, int64_t elem, bool i8, float scale, float (&x)[8]) {
    if (i8) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + elem);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu;
            x[i] = static_cast<float>(static_cast<int>(b) - static_cast<int>((b & 0x80u) << 1)) * scale;
        }
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(u[i]);
            x[2 * i + 1] = bf16_hi(u[i]);
        }
    }
}

__global__ void __launch_bounds__(kDsThreads) dense_simple_kernel(const DenseArgs a, int rows_per_cta, int tiles) {
    __shared__ float ks[kDsKeys][kHeadDim], vs[kDsKeys][kHeadDim];
    const int b = blockIdx.x / tiles, tile = blockIdx.x - b * tiles, h = blockIdx.y, tid = threadIdx.x;
    const int c0 = a.cu_rows[b], n = a.cu_rows[b + 1] - c0, L = a.cache_lens[b];
    if (n == 0 || (a.only_multi_row && n > 0 && n <= kDecodeMaxRows)) return;
    if (n < 0 || n > a.max_rows_per_seq || c0 < 0 || c0 + n > a.total_rows || L < n || L > a.max_cache_len ||
        !seq_rows_ok(a.cache, b, L, a.cache_tokens)) {
        if (tid == 0) atomicOr(a.err, kErrBadMetadata);
        return;
    }
    const int i0 = tile * rows_per_cta;
    if (i0 >= n) return;
    const int i = i0 + tid / a.G, g = tid % a.G;
    const bool live = tid < rows_per_cta * a.G && i < n;
    const int p = L - n + i;
    const int end = L - n + min(n, i0 + rows_per_cta);  // keys that some row of the CTA reads
    const int64_t qo = (static_cast<int64_t>(c0 + (live ? i : i0)) * a.H * a.G + h * a.G + g) * kHeadDim;
    uint32_t q[kHeadDim / 2];
    float o[kHeadDim], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < kHeadDim; d += 2) {
        q[d / 2] = *reinterpret_cast<const uint32_t*>(a.q + qo + d);
        o[d] = o[d + 1] = 0.f;
    }
    for (int t0 = 0; t0 < end; t0 += kDsKeys) {
        __syncthreads();
        for (int c = tid; c < kDsKeys * (kHeadDim / 8); c += kDsThreads) {
            const int t = t0 + c / (kHeadDim / 8), d = (c % (kHeadDim / 8)) * 8;
            float x[8] = {0.f}, y[8] = {0.f};
            if (t < end) {
                const int64_t first = block_row(a.cache, b, t & ~(kBlock - 1));
                if (first < 0) {
                    atomicOr(a.err, kErrBadMetadata);
                } else {
                    const int64_t row = (first + (t & (kBlock - 1))) * a.H + h;
                    ds_load8(a.k, row * kHeadDim + d, a.kv_int8, a.kv_int8 ? a.k_scale[row] : 1.f, x);
                    ds_load8(a.v, row * kHeadDim + d, a.kv_int8, a.kv_int8 ? a.v_scale[row] : 1.f, y);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ks[c / (kHeadDim / 8)][d + j] = x[j];
                vs[c / (kHeadDim / 8)][d + j] = y[j];
            }
        }
        __syncthreads();
        const int last = min(kDsKeys, p + 1 - t0);
        if (!live || last <= 0) continue;
        // a tile's scores and weights, then its sums, so that the running sums take one addition a tile
        float w[kDsKeys], top = m;
#pragma unroll
        for (int k = 0; k < kDsKeys; ++k) {
            float s2[2] = {0.f, 0.f};
#pragma unroll
            for (int d = 0; d < kHeadDim; d += 2) {
                s2[0] = fmaf(bf16_lo(q[d / 2]), ks[k][d], s2[0]);
                s2[1] = fmaf(bf16_hi(q[d / 2]), ks[k][d + 1], s2[1]);
            }
            w[k] = k < last ? (s2[0] + s2[1]) * a.scale_log2 : -INFINITY;
            top = fmaxf(top, w[k]);
        }
        const float f = exp2f(m - top);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kDsKeys; ++k) sum += w[k] = exp2f(w[k] - top);
        l = l * f + sum;
        m = top;
#pragma unroll
        for (int d = 0; d < kHeadDim; ++d) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < kDsKeys; ++k) x = k < last ? fmaf(w[k], vs[k][d], x) : x;
            o[d] = o[d] * f + x;
        }
    }
    if (!live) return;
    const float inv = 1.f / l;
#pragma unroll
    for (int d = 0; d < kHeadDim; d += 2) {
        if (a.out_bf16)
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + qo + d) = pack_bf16x2(o[d] * inv, o[d + 1] * inv);
        else
            *reinterpret_cast<float2*>(static_cast<float*>(a.out) + qo + d) = make_float2(o[d] * inv, o[d + 1] * inv);
    }
}

cudaError_t run_dense_simple(const DenseArgs& a, cudaStream_t stream) {
    const int rows = kDsThreads / a.G;
    const int tiles = (a.max_rows_per_seq + rows - 1) / rows;
    dense_simple_kernel<<<dim3(static_cast<unsigned>(a.num_seqs) * tiles, a.H), kDsThreads, 0, stream>>>(a, rows, tiles);
    return cudaGetLastError();
}

}  // namespace msa
