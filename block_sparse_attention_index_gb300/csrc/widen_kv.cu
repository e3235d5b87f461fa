// int8 key/value cache (PR #1388, native Metal family commit: keys and values
// cached as int8 with one scale per position and head), prompt chunks.
//
// In a long prompt chunk every 64-position block is kept by hundreds of
// (row, head) items, so widening the int8 tiles inside the attention repeats
// the same work that many times.  This pass widens the positions of every
// sequence the prompt-chunk attention reads once per call, into a contiguous
// bf16 copy in the workspace: the integers exactly (an int8 value has at most
// 8 significant bits, so bf16 holds it), the scales copied beside them in
// fp32.  The attention then loads bf16 tiles and multiplies the scores by the
// key scales and the weights by the value scales exactly as it does for the
// tiles it widens itself, so its results are those of the int8 cache.
//
// Layout: sequence b's copy starts at row  slot_b * slot_rows  (slot_b counts
// the widened sequences before b; slot_rows = max_cache_len rounded up to a
// whole block), rows [T', H, 128] bf16 for K and V and [H, T'] fp32 for the
// scales (head-major, so that a warp staging one head's scales for 32
// consecutive keys reads one 128-byte line).  Positions from L_b to the end of their 64-position block are
// written as zeros: keys past a row's position are masked, and a zero value
// keeps 0 x value out of the P V products.  Row starts per sequence go to
// `wide_starts` (0 for a sequence that is not widened, -1 for one past the
// slots the workspace holds, which the attention then rejects, or for one that another pass widens).
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace msa {

constexpr int kWidenThreads = 256;
constexpr int kWidenPos = 16;    // positions per work unit (a quarter block)
constexpr int kWidenBatch = 4;   // 16-byte chunks of K and of V a thread loads before it stores

// Byte i of w as a signed integer, then 4 bytes as 4 bf16 (two words; exact: at most 8 significant bits)
__device__ __forceinline__ float i8_at(uint32_t w, int i) {
    const int v = static_cast<int>((w >> (8 * i)) & 0xffu);
    return static_cast<float>(v - ((v & 0x80) << 1));
}
__device__ __forceinline__ uint2 widen_i8x4(uint32_t w) {
    return make_uint2(pack_bf16x2(i8_at(w, 0), i8_at(w, 1)), pack_bf16x2(i8_at(w, 2), i8_at(w, 3)));
}

// slot_of[b]: the slot of sequence b in this pass, or negative (-1 not widened, -2 past every pass's slots, -3 another
// pass widens it); CTA 0 writes the row starts.  The whole block calls it.
__device__ void widen_slots(const WidenArgs& a, int32_t* slot_of, int32_t* warp_tot) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = a.num_seqs;

    // ---- slots: thread t takes sequences [t per, (t + 1) per), then an exclusive block scan
    const int per = (B + kWidenThreads - 1) / kWidenThreads;
    const int b_lo = min(tid * per, B), b_hi = min(b_lo + per, B);
    int cnt = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int n = a.cu_rows[b + 1] - a.cu_rows[b];
        const int w = n >= 1 && !(a.only_multi_row && n <= kDecodeMaxRows);
        slot_of[b] = w;
        cnt += w;
    }
    int x = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    int excl = x - cnt;
    for (int i = 0; i < warp; ++i) excl += warp_tot[i];
    for (int b = b_lo; b < b_hi; ++b) {
        const int s = slot_of[b] ? excl++ : -1;
        // another pass widens it; past every pass's slots: more such sequences than the host counted
        slot_of[b] = s < 0 ? -1 : (s >= a.total_slots ? -2 : (s < a.first_slot || s >= a.first_slot + a.max_slots ? -3 : s - a.first_slot));
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int b = tid; b < B; b += kWidenThreads) {
            const int s = slot_of[b];
            a.wide_starts[b] = s == -1 ? 0 : (s < 0 ? -1 : static_cast<int64_t>(s) * a.slot_rows);
            if (s == -2) atomicOr(a.err, kErrBadMetadata);
        }
    }
}

__global__ void __launch_bounds__(kWidenThreads) widen_kv_kernel(const WidenArgs a) {
    extern __shared__ int32_t slot_of[];  // [num_seqs]: slot of sequence b, or -1 (not widened)
    __shared__ int32_t warp_tot[kWidenThreads / 32];
    const int tid = threadIdx.x, B = a.num_seqs;
    widen_slots(a, slot_of, warp_tot);

    // ---- units: (sequence, 16 positions), all heads, K and V; a block's positions past L_b are
    // written as zeros, so the units run to the end of the last block
    const int H = a.H;
    const int64_t wide_rows = static_cast<int64_t>(a.max_slots) * a.slot_rows;
    const int groups = a.slot_rows / kWidenPos;
    const int64_t units = static_cast<int64_t>(B) * groups;
    const int row_chunks = H * (kHeadDim / 16);  // 16-byte int8 chunks per position
    const int unit_chunks = kWidenPos * row_chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int b = static_cast<int>(u / groups), grp = static_cast<int>(u - static_cast<int64_t>(b) * groups);
        const int slot = slot_of[b];
        if (slot < 0) continue;
        const int L = a.cache_lens[b];
        const int t0 = grp * kWidenPos, tb = t0 & ~(kBlock - 1);  // first position, its block's
        if (L < 1 || L > a.max_cache_len || tb >= L) continue;  // the attention rejects such a sequence
        const int64_t brow = seq_rows_ok(a.cache, b, L, a.cache_tokens) ? block_row(a.cache, b, tb) : -1;
        if (brow < 0 && tid == 0 && t0 == tb) atomicOr(a.err, kErrBadMetadata);  // the block is written as zeros
        const int64_t src = brow < 0 ? 0 : brow + (t0 - tb);  // a block's rows are contiguous (a page holds whole blocks)
        const int64_t dst = static_cast<int64_t>(slot) * a.slot_rows + t0;
        const int live_rows = brow < 0 ? 0 : max(0, min(kWidenPos, L - t0));
        const uint8_t* k8 = a.k8 + src * H * kHeadDim;
        const uint8_t* v8 = a.v8 + src * H * kHeadDim;
        uint16_t* kw = a.kw + dst * H * kHeadDim;
        uint16_t* vw = a.vw + dst * H * kHeadDim;
        for (int c0 = tid; c0 < unit_chunks; c0 += kWidenBatch * kWidenThreads) {
            uint4 kx[kWidenBatch], vx[kWidenBatch];  // every load of the batch in flight before a store
#pragma unroll
            for (int j = 0; j < kWidenBatch; ++j) {
                const int c = c0 + j * kWidenThreads;
                const bool live = c < live_rows * row_chunks;
                kx[j] = live ? ld_stream_v4(k8 + c * 16) : make_uint4(0, 0, 0, 0);
                vx[j] = live ? ld_stream_v4(v8 + c * 16) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < kWidenBatch; ++j) {
                const int c = c0 + j * kWidenThreads;
                if (c >= unit_chunks) break;
                const uint2 k0 = widen_i8x4(kx[j].x), k1 = widen_i8x4(kx[j].y), k2 = widen_i8x4(kx[j].z),
                            k3 = widen_i8x4(kx[j].w);
                const uint2 v0 = widen_i8x4(vx[j].x), v1 = widen_i8x4(vx[j].y), v2 = widen_i8x4(vx[j].z),
                            v3 = widen_i8x4(vx[j].w);
                uint4* kd = reinterpret_cast<uint4*>(kw + static_cast<int64_t>(c) * 16);
                uint4* vd = reinterpret_cast<uint4*>(vw + static_cast<int64_t>(c) * 16);
                kd[0] = make_uint4(k0.x, k0.y, k1.x, k1.y);
                kd[1] = make_uint4(k2.x, k2.y, k3.x, k3.y);
                vd[0] = make_uint4(v0.x, v0.y, v1.x, v1.y);
                vd[1] = make_uint4(v2.x, v2.y, v3.x, v3.y);
            }
        }
        for (int c = tid; c < kWidenPos * H; c += kWidenThreads) {  // scales head-major: [H][rows]
            const bool live = c < live_rows * H;
            const int pos = c / H, h = c - pos * H;
            const int64_t o = static_cast<int64_t>(h) * wide_rows + dst + pos;
            a.ksw[o] = live ? a.k_scale[src * H + c] : 0.f;
            a.vsw[o] = live ? a.v_scale[src * H + c] : 0.f;
        }
    }
}

// The same for outputs of 16 bits in the dense attention: f16 values with the scales in them, over a power of two for
// each 64-position block and head (so that nothing overflows).  A scale down to 2^-22 of that power of two keeps f16's
// 11 bits: a key or value is off by 2^-11 of itself at most.  Below, small codes have fewer bits or none (a token whose
// scale is 2^22 times its neighbours', which the rows before it must not notice).  fac[h][block] = (the power of two to
// multiply key products by, its lowest bit set, 2^-23 of it, if some key or value of the block has lost bits, and
// *any_lost too; the one to multiply the value sums by, 0 for values that are all 0).  CTA: a block, all heads.
__global__ void __launch_bounds__(kWidenThreads) widen_f16_kernel(const WidenArgs a, float2* fac, uint32_t* any_lost) {
    extern __shared__ int32_t slot_of[];  // [num_seqs]
    __shared__ int32_t warp_tot[kWidenThreads / 32];
    __shared__ float scale[2][kBlock * 8];  // key and value scales of the block, [position][head]
    __shared__ float top[2][8];             // their powers of two
    __shared__ bool zero[2][8], lost[2][8]; // all scales are 0; some scale is too far below
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.num_seqs, H = a.H;
    widen_slots(a, slot_of, warp_tot);
    const int blocks = a.slot_rows / kBlock;
    const int64_t wide_blocks = static_cast<int64_t>(a.max_slots) * blocks;
    const int row_chunks = H * (kHeadDim / 16), chunks = kBlock * row_chunks;
    for (int64_t u = blockIdx.x; u < static_cast<int64_t>(B) * blocks; u += gridDim.x) {
        const int b = static_cast<int>(u / blocks), blk = static_cast<int>(u - static_cast<int64_t>(b) * blocks);
        const int slot = slot_of[b];
        if (slot < 0) continue;
        const int L = a.cache_lens[b], t0 = blk * kBlock;
        if (L < 1 || L > a.max_cache_len || t0 >= L) continue;  // the attention rejects such a sequence
        const int64_t src = seq_rows_ok(a.cache, b, L, a.cache_tokens) ? block_row(a.cache, b, t0) : -1;
        if (src < 0 && tid == 0) atomicOr(a.err, kErrBadMetadata);  // the block is written as zeros
        const int live = src < 0 ? 0 : min(kBlock, L - t0);
        __syncthreads();  // the last block's scales are done with
        for (int c = tid; c < kBlock * H; c += kWidenThreads) {
            scale[0][c] = c < live * H ? a.k_scale[src * H + c] : 0.f;
            scale[1][c] = c < live * H ? a.v_scale[src * H + c] : 0.f;
        }
        __syncthreads();
        for (int c = warp; c < 2 * H; c += kWidenThreads / 32) {  // a warp a (kind, head): the largest finite scale
            const int kind = c / H, h = c - kind * H;
            float most = 0.f, least = INFINITY;  // (of the scales that are not zero)
            for (int pos = lane; pos < kBlock; pos += 32) {
                const float x = fabsf(scale[kind][pos * H + h]);
                if (x < INFINITY) most = fmaxf(most, x);
                if (x > 0.f) least = fminf(least, x);
            }
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(most));  // (positive: ordered as their bits)
            least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(least)));
            // the next power of two, in [2^-110, 2^127]: 256 / it and it / 256 are normal numbers
            const uint32_t bits = (m + 0x007FFFFFu) & 0x7F800000u;
            const float power = __uint_as_float(min(max(bits, 17u << 23), 0x7F000000u));
            if (lane == 0) {
                top[kind][h] = power;
                zero[kind][h] = m == 0u;
                lost[kind][h] = least < power * 2.384185791015625e-7f;  // 2^-22
            }
        }
        __syncthreads();
        const int64_t dst = (static_cast<int64_t>(slot) * blocks + blk) * kBlock;
        if (tid < H) {
            const uint32_t bad = lost[0][tid] || lost[1][tid];
            fac[tid * wide_blocks + dst / kBlock] = make_float2(__uint_as_float(__float_as_uint(top[0][tid] / 256.f) | bad),
                                                                zero[1][tid] ? 0.f : top[1][tid] / 256.f);
            if (bad) *any_lost = 1u;
        }
        const uint8_t* in[2] = {a.k8 + src * H * kHeadDim, a.v8 + src * H * kHeadDim};
        uint16_t* out[2] = {a.kw + dst * H * kHeadDim, a.vw + dst * H * kHeadDim};
        for (int c0 = tid; c0 < chunks; c0 += kWidenBatch * kWidenThreads) {
            uint4 x[2][kWidenBatch];  // every load of the batch in flight before a store
#pragma unroll
            for (int j = 0; j < kWidenBatch; ++j) {
                const int c = c0 + j * kWidenThreads;
#pragma unroll
                for (int kind = 0; kind < 2; ++kind)
                    x[kind][j] = c < live * row_chunks ? ld_stream_v4(in[kind] + c * 16) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < kWidenBatch; ++j) {
                const int c = c0 + j * kWidenThreads;
                if (c >= chunks) break;
                const int head = c / (kHeadDim / 16) % H;
#pragma unroll
                for (int kind = 0; kind < 2; ++kind) {
                    const float f = scale[kind][c / (kHeadDim / 16)] * (256.f / top[kind][head]);
                    const uint32_t w[4] = {x[kind][j].x, x[kind][j].y, x[kind][j].z, x[kind][j].w};
                    uint32_t y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const __half2 v = __floats2half2_rn(i8_at(w[i], 2 * e) * f, i8_at(w[i], 2 * e + 1) * f);
                            y[2 * i + e] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                    uint4* d = reinterpret_cast<uint4*>(out[kind] + static_cast<int64_t>(c) * 16);
                    d[0] = make_uint4(y[0], y[1], y[2], y[3]);
                    d[1] = make_uint4(y[4], y[5], y[6], y[7]);
                }
            }
        }
    }
}

cudaError_t run_widen_f16(const WidenArgs& a, float2* fac, uint32_t* any_lost, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(a.num_seqs) * (a.slot_rows / kBlock);
    const int64_t cap = 4 * static_cast<int64_t>(device_sm_count());
    const int grid = static_cast<int>(units < cap ? (units > 0 ? units : 1) : cap);
    widen_f16_kernel<<<grid, kWidenThreads, static_cast<size_t>(a.num_seqs) * sizeof(int32_t), stream>>>(a, fac, any_lost);
    return cudaGetLastError();
}

cudaError_t run_widen_kv(const WidenArgs& a, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(a.num_seqs) * (a.slot_rows / kWidenPos);
    const int64_t cap = 4 * static_cast<int64_t>(device_sm_count());
    const int grid = static_cast<int>(units < cap ? (units > 0 ? units : 1) : cap);
    const size_t smem = static_cast<size_t>(a.num_seqs) * sizeof(int32_t);
    widen_kv_kernel<<<grid, kWidenThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace msa
