// Cache writer: rotary positions on the new rows' queries, keys and index
// keys, and the store of keys, values and index keys into the caches.
//   angle_j = 2 pi frac(x turns_j / 2^64),  x = the row's position on axis_j
//   y_a = x_a cos - x_b sin,  y_b = x_b cos + x_a sin      for the pair (a, b) of j
//   bf16 cache: y rounded;  int8: scale = max |y| / 127, codes = rint(y / scale)
// x turns_j is a 64-bit product modulo one turn, so the phase of a far
// position is as exact as a near one's (fp32 angles lose 0.1 rad at 2^21);
// its upper 32 bits, as a signed number of half turns, feed sincospi.
//
// Bound by memory: every value is read once and written once.  A CTA takes a
// few rows, computes their cosines and sines once into shared memory (all
// heads of a row share them) and then walks the rows' 16-byte chunks of q, k,
// v, iq and ik.  16 lanes (8 for the 64-dimension index heads) hold one head,
// 8 values each, so the rotation's partner in the half-split pairing is the
// same element of another lane (one shuffle a word) and a head's maximum for
// the int8 scale is four shuffles.
#include "common.cuh"
#include "internal.h"

namespace msa {

constexpr int kApThreads = 256;
constexpr int kApRows = 8;    // most rows a CTA takes at a time
constexpr int kApPairs = kHeadDim / 2 + kIndexDim / 2;
constexpr int kApBatch = 4;   // chunks a thread loads before it stores any

struct ApRow {
    int32_t r;         // row, or -1: not stored
    int32_t pos;
    int64_t cache;     // cache row, or -1
};

// One 8-value chunk of a head, as it lies in q, k, v, iq or ik.
struct ApChunk {
    int kind;  // 0 q, 1 k, 2 v, 3 iq, 4 ik, -1 none
    int head, d0;
};

__device__ __forceinline__ ApChunk ap_chunk(int c, int nq, int nk, int niq, int nik) {
    ApChunk x;
    x.kind = 0;
    if (c >= nq) { c -= nq; x.kind = 1;
        if (c >= nk) { c -= nk; x.kind = 2;
            if (c >= nk) { c -= nk; x.kind = 3;
                if (c >= niq) { c -= niq; x.kind = c < nik ? 4 : -1; } } } }
    const bool index = x.kind >= 3;
    x.head = index ? c >> 3 : c >> 4;
    x.d0 = (index ? c & 7 : c & 15) * 8;
    return x;
}

__global__ void __launch_bounds__(kApThreads) append_cache_kernel(const AppendArgs a, int rows_per_cta) {
    __shared__ ApRow row_of[kApRows];
    __shared__ float2 turn[kApRows][kApPairs];  // (cos, sin) of the head pairs, then of the index pairs
    const int tid = threadIdx.x, lane = tid & 31;
    const int H = a.H, HG = a.H * a.G;
    const int nq = a.q ? HG * 16 : 0, nk = H * 16, niq = a.iq ? H * 8 : 0, nik = a.ik ? a.KH * 8 : 0;
    const int chunks = nq + 2 * nk + niq + nik;
    const int pairs = a.rope_dim / 2, ipairs = a.rope_index_dim / 2;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * rows_per_cta; first < a.total_rows;
         first += static_cast<int64_t>(gridDim.x) * rows_per_cta) {
        __syncthreads();  // the last rows' chunks are done with the shared arrays
        if (tid < rows_per_cta) {
            ApRow x{-1, 0, -1};
            const int64_t r = first + tid;
            if (r < a.total_rows) {
                int lo = 0, hi = a.num_seqs;  // largest b with cu_rows[b] <= r
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (a.cu_rows[mid] <= r) lo = mid; else hi = mid;
                }
                const int b = lo, c0 = a.cu_rows[b], c1 = a.cu_rows[b + 1], n = c1 - c0, L = a.cache_lens[b];
                if (r >= c0 && r < c1) {
                    if (n > a.max_rows_per_seq || c0 < 0 || c1 > a.total_rows || L < n || L > a.max_cache_len ||
                        !seq_rows_ok(a.cache, b, L, a.cache_tokens)) {
                        atomicOr(a.err, kErrBadMetadata);
                    } else {
                        x.r = static_cast<int>(r);
                        x.pos = L - n + static_cast<int>(r - c0);
                        const int64_t first_row = block_row(a.cache, b, x.pos & ~(kBlock - 1));
                        if (first_row < 0) atomicOr(a.err, kErrBadMetadata);  // page outside the pool
                        else x.cache = first_row + (x.pos & (kBlock - 1));
                    }
                } else if (r < c0 || b + 1 < a.num_seqs) {
                    atomicOr(a.err, kErrBadMetadata);  // cu_rows not ascending (rows past the last sequence are nobody's)
                }
            }
            row_of[tid] = x;
        }
        __syncthreads();
        for (int c = tid; c < rows_per_cta * (pairs + ipairs); c += kApThreads) {
            const int i = c / (pairs + ipairs), j = c - i * (pairs + ipairs);
            const ApRow x = row_of[i];
            if (x.r < 0) continue;
            const bool index = j >= pairs;
            const int k = index ? j - pairs : j;
            const int32_t* axis = index ? a.index_axis : a.axis;
            int ax = axis ? axis[k] : 0;
            if (ax < 0 || ax >= a.axes) {
                atomicOr(a.err, kErrBadMetadata);
                ax = 0;
            }
            const int64_t where = a.positions ? a.positions[static_cast<int64_t>(ax) * a.total_rows + x.r] : x.pos;
            const uint64_t phase = static_cast<uint64_t>(where) * (index ? a.index_turns : a.turns)[k];
            float s, co;
            sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &co);  // 2^-31
            turn[i][index ? kHeadDim / 2 + k : k] = make_float2(co, s);
        }
        __syncthreads();
        const int total = rows_per_cta * chunks;
        // every lane of a warp runs the same number of passes (the shuffles need them all)
        for (int base = tid - lane; base < total; base += kApBatch * kApThreads) {
            uint4 w[kApBatch];
            ApChunk x[kApBatch];
            int row[kApBatch];
#pragma unroll
            for (int u = 0; u < kApBatch; ++u) {
                const int c = base + u * kApThreads + lane;
                row[u] = c < total ? c / chunks : 0;
                x[u] = ap_chunk(c - row[u] * chunks, nq, nk, niq, nik);
                if (c >= total || row_of[row[u]].r < 0) x[u].kind = -1;
                w[u] = make_uint4(0, 0, 0, 0);
                if (x[u].kind >= 0) {
                    const int64_t r = row_of[row[u]].r;
                    const uint16_t* src = x[u].kind == 0 ? a.q + r * a.q_stride
                                        : x[u].kind == 1 ? a.k + r * a.k_stride
                                        : x[u].kind == 2 ? a.v + r * a.v_stride
                                        : x[u].kind == 3 ? a.iq + r * a.iq_stride : a.ik + r * a.ik_stride;
                    w[u] = *reinterpret_cast<const uint4*>(src + x[u].head * (x[u].kind >= 3 ? kIndexDim : kHeadDim) + x[u].d0);
                }
            }
#pragma unroll
            for (int u = 0; u < kApBatch; ++u) {
                if (base + u * kApThreads >= total) break;  // uniform over the warp
                const int kind = x[u].kind;
                const bool index = kind >= 3;
                const int dim = kind == 2 || kind < 0 ? 0 : (index ? a.rope_index_dim : a.rope_dim);
                const float2* cs = &turn[row[u]][index ? kHeadDim / 2 : 0];
                uint32_t mine[4] = {w[u].x, w[u].y, w[u].z, w[u].w}, other[4];
                const int step = dim / 16;  // lanes from a value to its partner
                const bool lower = x[u].d0 < dim / 2;
                const int partner = lane + (dim == 0 || x[u].d0 >= dim ? 0 : (lower ? step : -step));
#pragma unroll
                for (int e = 0; e < 4; ++e) other[e] = __shfl_sync(0xffffffffu, mine[e], partner);
                float y[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[2 * e] = bf16_lo(mine[e]);
                    y[2 * e + 1] = bf16_hi(mine[e]);
                }
                const bool turned = x[u].d0 < dim;
                if (turned && a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 t = cs[x[u].d0 / 2 + e];
                        const float p0 = y[2 * e], p1 = y[2 * e + 1];
                        y[2 * e] = p0 * t.x - p1 * t.y;
                        y[2 * e + 1] = p1 * t.x + p0 * t.y;
                    }
                } else if (turned) {
                    const int j0 = lower ? x[u].d0 : x[u].d0 - dim / 2;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = cs[j0 + e];
                        const float z = e & 1 ? bf16_hi(other[e >> 1]) : bf16_lo(other[e >> 1]);
                        y[e] = lower ? y[e] * t.x - z * t.y : y[e] * t.x + z * t.y;
                    }
                }
                const int64_t cache = kind < 0 ? -1 : row_of[row[u]].cache;
                if (a.kv_int8) {  // the 16 lanes of a key or value head
                    uint32_t top = 0;  // largest magnitude as bits: a NaN counts as larger than infinity
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (kind == 1 || kind == 2) {
                        if (cache < 0) continue;
                        const float scale = __fdiv_rn(__uint_as_float(top), 127.f);
                        uint32_t code[2] = {0u, 0u};
                        if (scale > 0.f && scale < INFINITY) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float q = fminf(fmaxf(rintf(__fdiv_rn(y[e], scale)), -127.f), 127.f);
                                code[e >> 2] |= (static_cast<uint32_t>(static_cast<int>(q)) & 0xffu) << (8 * (e & 3));
                            }
                        }
                        const int64_t o = cache * H + x[u].head;
                        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kind == 1 ? a.k_cache : a.v_cache) + o * kHeadDim +
                                                  x[u].d0) = make_uint2(code[0], code[1]);
                        if (x[u].d0 == 0) (kind == 1 ? a.k_scale : a.v_scale)[o] = scale;
                        continue;
                    }
                }
                if (kind < 0) continue;
                const int64_t r = row_of[row[u]].r;
                uint16_t* dst;
                if (kind == 0) {
                    dst = a.q_out + (r * HG + x[u].head) * kHeadDim;
                } else if (kind == 3) {
                    dst = a.iq_out + (r * H + x[u].head) * kIndexDim;
                } else {
                    if (cache < 0) continue;
                    dst = kind == 4 ? a.ik_cache + (cache * a.KH + x[u].head) * kIndexDim
                                    : static_cast<uint16_t*>(kind == 1 ? a.k_cache : a.v_cache) + (cache * H + x[u].head) * kHeadDim;
                }
                if (turned)
                    w[u] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                      pack_bf16x2(y[6], y[7]));
                *reinterpret_cast<uint4*>(dst + x[u].d0) = w[u];
            }
        }
    }
}

cudaError_t run_append_cache(const AppendArgs& a, cudaStream_t stream) {
    const int sms = device_sm_count();
    int rows = a.total_rows / (4 * sms);  // few rows: one to a CTA
    rows = rows < 1 ? 1 : (rows > kApRows ? kApRows : rows);
    const int64_t need = (static_cast<int64_t>(a.total_rows) + rows - 1) / rows;
    const int64_t cap = 8 * static_cast<int64_t>(sms);
    append_cache_kernel<<<static_cast<unsigned>(need < cap ? need : cap), kApThreads, 0, stream>>>(a, rows);
    return cudaGetLastError();
}

}  // namespace msa
