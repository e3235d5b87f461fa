// Cache writer: rotary positions on the new rows' queries, keys and index
// keys, and the store of keys, values and index keys into the caches.
//   angle_j = 2 pi frac(x turns_j / 2^64),  x = the row's position on axis_j
//   y_a = x_a cos - x_b sin,  y_b = x_b cos + x_a sin      for the pair (a, b) of j
//   bf16 cache: y rounded;  int8: scale = max |y| / 127, codes = rint(y / scale)
//   int8 index keys: the least e with max |y| <= 127 2^e, codes = rint(y 2^-e): a power of two, so that a code read back
//   is a bf16 value exactly.  A head with a value so near to a half that fp32 may be on its other side (1.5 % of them), or
//   one past 32 bits' range, is rotated again in 64 bits when the CTA's rows are done: codes and exponents are whole numbers that
//   decide which blocks are kept, and are the definition's, not one of two neighbours (as int8 keys' codes may be).
// x turns_j is a 64-bit product modulo one turn, so the phase of a far
// position is as exact as a near one's (fp32 angles lose 0.1 rad at 2^21);
// its upper 32 bits, as a signed number of half turns, feed sincospi.
//
// Bound by memory: every value is read once and written once; few rows are
// bound by the chain of dependent loads (metadata, page number).  A CTA takes
// a few rows, sends off its first loads, finds the rows' cache rows (one
// thread a sequence where all fit, so one load latency instead of a search's),
// computes their cosines and sines once into shared memory (all heads of a row
// share them) and walks the rows' heads.  A warp takes two heads of q, k or v
// at a time, or four of the 64-dimension index heads, 8 values (16 bytes) a
// lane.  The query heads, most of the data, have a short loop of their own (a
// lane keeps its cosines and sines in registers for the heads of a row); one
// loop for all kinds was bound by its instructions, 240 a warp's 512 bytes.  The
// rotation's partner in the half-split pairing is the same element of another
// lane (one shuffle a word) and a head's maximum for the int8 scale is four
// shuffles.  Codes come from a
// product with 1 / scale, and from the exact quotient in the (rare) heads with
// a value so near a half that the product could round the other way.
//
// Measured: 4,096 rows of 4 x 16 heads into an int8 cache, 45 us (155 MB: 3.4 TB/s, 55 % of the issue slots taken; four
// CTAs an SM instead of three spill: 51 us); 8 paged rows, 8.5 us, of which an empty launch is about 7.5.  With index
// keys of 8 bits 44 us and the same (their 64-bit rotations; 40 without).
#include "common.cuh"
#include "internal.h"

namespace msa {

constexpr int kApThreads = 256;
constexpr int kApWarps = kApThreads / 32;
constexpr int kApRows = 16;   // most rows a CTA takes at a time
constexpr int kApPairs = kHeadDim / 2 + kIndexDim / 2;
constexpr int kApBatch = 4;   // pairs of query heads that a warp loads before it stores any
constexpr float kApNear = 1.f / 8192;  // index codes: how near to a half counts as near
constexpr int kApCheckRows = 256;  // up to so many rows CTA 0 alone reports bad metadata (and stores the error word)

struct ApRow {
    int32_t r;         // row, or -1: not stored
    int32_t pos;
    int64_t cache;     // cache row, or -1
};

// What sequence b gives its row r: the row's position and cache row; bits of the error word if something is wrong.
__device__ __forceinline__ uint32_t ap_place(const AppendArgs& a, int b, int c0, int c1, int L, int64_t r, ApRow& x) {
    const int n = c1 - c0;
    if (n > a.max_rows_per_seq || c0 < 0 || c1 > a.total_rows || L < n || L > a.max_cache_len ||
        !seq_rows_ok(a.cache, b, L, a.cache_tokens))
        return kErrBadMetadata;
    x.r = static_cast<int>(r);
    x.pos = L - n + static_cast<int>(r - c0);
    const int64_t first = block_row(a.cache, b, x.pos & ~(kBlock - 1));
    if (first < 0) return kErrBadMetadata;  // page outside the pool
    x.cache = first + (x.pos & (kBlock - 1));
    return 0;
}

// The same for row r by a search of its sequence.
__device__ uint32_t ap_find(const AppendArgs& a, int64_t r, ApRow& x) {
    int lo = 0, hi = a.num_seqs;  // largest b with cu_rows[b] <= r
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_rows[mid] <= r) lo = mid; else hi = mid;
    }
    const int c0 = a.cu_rows[lo], c1 = a.cu_rows[lo + 1];
    if (r >= c0 && r < c1) return ap_place(a, lo, c0, c1, a.cache_lens[lo], r, x);
    // rows past the last sequence are nobody's; else cu_rows does not ascend
    return r < c0 || lo + 1 < a.num_seqs ? kErrBadMetadata : 0;
}

// 8 codes of the lane's values (scale > 0 and finite): rint(y / scale), clamped to [-127, 127].
__device__ __forceinline__ uint2 ap_codes(const float (&y)[8], float scale) {
    const float inv = 1.f / scale;
    float t[8], near = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = y[e] * inv;
        t[e] = q + 12582912.f;  // 1.5 2^23: rounds to an integer, whose two's complement is in the low bits
        near = fmaxf(near, fabsf(q - (t[e] - 12582912.f)));
    }
    // y inv is within 127 2^-22 of the quotient, which near a half may round the other way; a subnormal scale may be
    // too coarse for |y| <= 127 scale
    if (near > 0.4999f || scale < 1.1754944e-38f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = fminf(fmaxf(rintf(__fdiv_rn(y[e], scale)), -127.f), 127.f) + 12582912.f;
    }
    uint32_t c[2];
#pragma unroll
    for (int w = 0; w < 2; ++w)
        c[w] = __byte_perm(__byte_perm(__float_as_uint(t[4 * w]), __float_as_uint(t[4 * w + 1]), 0x0040),
                           __byte_perm(__float_as_uint(t[4 * w + 2]), __float_as_uint(t[4 * w + 3]), 0x0040), 0x5410);
    return make_uint2(c[0], c[1]);
}

// The power of two of an index head from its largest magnitude as bits (not finite: -128): 127 is 1.984375 2^6.
__device__ __forceinline__ int ap_index_exp(uint32_t top) {
    if (top >= 0x7f800000u) return -128;
    return max(static_cast<int>(top >> 23) - 133 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0), -126);
}

// 8 codes of y 2^-e, which is exact and at most 127.
__device__ __forceinline__ uint2 ap_index_codes(const float (&y)[8], int e) {
    const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __float_as_uint(fmaf(y[i], f, 12582912.f));  // 1.5 2^23: an integer in the low bits
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
    return make_uint2(w[0], w[1]);
}

// An index head's codes and exponent from a rotation in 64 bits: a warp, two values a lane.
__device__ __forceinline__ void ap_index_again(const AppendArgs& a, const ApRow& row, int head, int lane) {
    const uint16_t* src = a.ik + row.r * a.ik_stride + head * kIndexDim;
    const int half = a.rope_index_dim / 2;
    double y[2];
    unsigned long long top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int d = 2 * lane + i;
        y[i] = __uint_as_float(static_cast<uint32_t>(src[d]) << 16);
        if (d < a.rope_index_dim) {
            const bool lower = a.interleaved ? i == 0 : d < half;
            const int pair = a.interleaved ? lane : (lower ? d : d - half), other = a.interleaved ? d ^ 1 : (lower ? d + half : d - half);
            int ax = a.index_axis ? a.index_axis[pair] : 0;
            if (ax < 0 || ax >= a.axes) ax = 0;
            const int64_t where = a.positions ? a.positions[static_cast<int64_t>(ax) * a.total_rows + row.r] : row.pos;
            const uint64_t phase = static_cast<uint64_t>(where) * a.index_turns[pair];
            const double z = __uint_as_float(static_cast<uint32_t>(src[other]) << 16);
            double s, c;
            sincospi(static_cast<double>(static_cast<int64_t>(phase)) * 1.0842021724855044e-19, &s, &c);  // 2^-63
            y[i] = y[i] * c + (lower ? -z : z) * s;
        }
        top = max(top, static_cast<unsigned long long>(__double_as_longlong(fabs(y[i]))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7FF0000000000000ull;
    const int e = finite ? max(static_cast<int>(top >> 52) - 1029 + ((top & 0xFFFFFFFFFFFFFull) > 0xFC00000000000ull ? 1 : 0), -126) : -128;
    const double f = __longlong_as_double(static_cast<long long>(1023 - e) << 52);
    const uint32_t lo = finite ? __double2int_rn(y[0] * f) & 0xff : 0, hi = finite ? __double2int_rn(y[1] * f) & 0xff : 0;
    const int64_t o = row.cache * a.KH + head;
    *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.ik_cache) + o * kIndexDim + 2 * lane) = static_cast<uint16_t>(lo | hi << 8);
    if (lane == 0) a.ik_exp[o] = static_cast<int8_t>(e);
}

template <bool kCodes>
__global__ void __launch_bounds__(kApThreads, 3) append_cache_kernel(const AppendArgs a, int rows_per_cta, int team) {
    __shared__ int again;  // index heads that are to be rotated in 64 bits, and which: 8 i + head
    __shared__ uint16_t again_of[kCodes ? kApRows * 8 : 1];
    __shared__ ApRow row_of[kApRows];
    __shared__ __align__(16) float2 turn[kApRows][kApPairs];  // (cos, sin) of the head pairs, then of the index pairs
    __shared__ uint32_t err;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int member = warp % team, teams = kApWarps / team, my_team = warp / team;  // `team` warps share a row
    const int H = a.H, HG = a.H * a.G;
    const bool check_all = a.total_rows <= kApCheckRows;
    // of a row: pairs of query heads, and the other tasks: pairs of key heads, of value heads, fours of index heads
    const int tq = a.q ? (HG + 1) / 2 : 0, tk = (H + 1) / 2, ti = a.iq ? (H + 3) / 4 : 0, tx = a.ik ? (a.KH + 3) / 4 : 0;
    const int others = 2 * tk + ti + tx;
    const int pairs = a.rope_dim / 2, ipairs = a.rope_index_dim / 2;
    if (tid == 0) err = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * rows_per_cta; first < a.total_rows;
         first += static_cast<int64_t>(gridDim.x) * rows_per_cta) {
        const int rows = static_cast<int>(min(static_cast<int64_t>(rows_per_cta), a.total_rows - first));
        // the warp's query heads of a row: load batch t0 .. (also ahead of the metadata, for the first row)
        const int qhead = lane >> 4, d0 = (lane & 15) * 8;
        auto load_q = [&](int i, int t0, uint4 (&w)[kApBatch]) {
            const uint16_t* src = a.q + (first + i) * a.q_stride + d0;
#pragma unroll
            for (int u = 0; u < kApBatch; ++u) {
                const int head = 2 * (t0 + u * team) + qhead;
                w[u] = head < HG ? *reinterpret_cast<const uint4*>(src + head * kHeadDim) : make_uint4(0, 0, 0, 0);
            }
        };
        // task t of the others: 1 k, 2 v, 3 iq, 4 ik (the same for the warp), the lane's head and first dimension
        auto other_task = [&](int t, int& k, int& head, int& at) {
            int c = t;
            k = 1;
            if (c >= tk) { c -= tk; k = 2;
                if (c >= tk) { c -= tk; k = 3;
                    if (c >= ti) { c -= ti; k = 4; } } }
            head = k >= 3 ? 4 * c + (lane >> 3) : 2 * c + (lane >> 4);
            at = (k >= 3 ? lane & 7 : lane & 15) * 8;
            return head < (k == 4 ? a.KH : H);  // a head that is not there goes along and stores nothing
        };
        auto load_other = [&](int i, int t) {
            int k, head, at;
            if (!other_task(t, k, head, at)) return make_uint4(0, 0, 0, 0);
            const int64_t r = first + i;
            const uint16_t* src = k == 1 ? a.k + r * a.k_stride
                                : k == 2 ? a.v + r * a.v_stride
                                : k == 3 ? a.iq + r * a.iq_stride : a.ik + r * a.ik_stride;
            return *reinterpret_cast<const uint4*>(src + head * (k >= 3 ? kIndexDim : kHeadDim) + at);
        };
        const int other0 = team - 1 - member;  // from the last warp on, which has the fewest query heads
        uint4 w[kApBatch], ov = make_uint4(0, 0, 0, 0);
        if (my_team < rows) {
            if (member < tq) load_q(my_team, member, w);
            if (other0 < others) ov = load_other(my_team, other0);
        }
        __syncthreads();  // the last rows' tasks are done with the shared arrays
        if (kCodes && tid == 0) again = 0;
        if (a.num_seqs <= kApThreads) {
            if (tid < rows_per_cta) row_of[tid] = ApRow{-1, 0, -1};
            int c0 = 0, c1 = 0, L = 0;
            if (tid < a.num_seqs) {
                c0 = a.cu_rows[tid];
                c1 = a.cu_rows[tid + 1];
                L = a.cache_lens[tid];
            }
            __syncthreads();
            uint32_t bad = tid < a.num_seqs && c1 < c0 ? kErrBadMetadata : 0u;
            for (int64_t r = max(static_cast<int64_t>(c0), first); r < min(static_cast<int64_t>(c1), first + rows); ++r) {
                ApRow x{-1, 0, -1};
                bad |= ap_place(a, tid, c0, c1, L, r, x);
                row_of[r - first] = x;
            }
            if (bad) atomicOr(&err, bad);
        } else if (tid < rows_per_cta) {
            ApRow x{-1, 0, -1};
            const uint32_t bad = tid < rows ? ap_find(a, first + tid, x) : 0u;
            if (bad) atomicOr(&err, bad);
            row_of[tid] = x;
        }
        __syncthreads();
        for (int c = tid; c < rows * (pairs + ipairs); c += kApThreads) {
            const int i = c / (pairs + ipairs), j = c - i * (pairs + ipairs);
            const ApRow x = row_of[i];
            if (x.r < 0) continue;
            const bool index = j >= pairs;
            const int k = index ? j - pairs : j;
            const int32_t* axis = index ? a.index_axis : a.axis;
            int ax = axis ? axis[k] : 0;
            if (ax < 0 || ax >= a.axes) {
                atomicOr(&err, kErrBadMetadata);
                ax = 0;
            }
            const int64_t where = a.positions ? a.positions[static_cast<int64_t>(ax) * a.total_rows + x.r] : x.pos;
            const uint64_t phase = static_cast<uint64_t>(where) * (index ? a.index_turns : a.turns)[k];
            float s, co;
            sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &co);  // 2^-31
            turn[i][index ? kHeadDim / 2 + k : k] = make_float2(co, s);
        }
        __syncthreads();

        for (int i = my_team; i < rows; i += teams) {
            const ApRow row = row_of[i];
            const int64_t r = row.r;
            if (r >= 0) {  // ---- query heads
                const int half = a.rope_dim / 2, step = a.rope_dim / 16;
                const bool turned = d0 < a.rope_dim, lower = d0 < half;
                // the lane's cosines and (signed) sines, of its 8 values; interleaved: of its 4 pairs
                float2 co[4], si[4];
                if (turned) {
                    const float4* t = reinterpret_cast<const float4*>(&turn[i][a.interleaved ? d0 / 2 : (lower ? d0 : d0 - half)]);
                    const float sign = lower || a.interleaved ? -1.f : 1.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 v = t[a.interleaved ? e >> 1 : e];
                        if (a.interleaved) {
                            co[e] = e & 1 ? make_float2(v.z, v.z) : make_float2(v.x, v.x);
                            si[e] = e & 1 ? make_float2(-v.w, v.w) : make_float2(-v.y, v.y);
                        } else {
                            co[e] = make_float2(v.x, v.z);
                            si[e] = make_float2(sign * v.y, sign * v.w);
                        }
                    }
                }
                const int partner = turned && !a.interleaved ? lane + (lower ? step : -step) : lane;
                uint16_t* dst = a.q_out + r * HG * kHeadDim + d0;
                for (int t = member; t < tq; t += kApBatch * team) {
                    if (t > member) load_q(i, t, w);
#pragma unroll
                    for (int u = 0; u < kApBatch; ++u) {
                        if (t + u * team >= tq) break;
                        const int head = 2 * (t + u * team) + qhead;
                        uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w}, z[4];
                        if (a.rope_dim > 0) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)  // the partner's values: another lane's, or the pair's other half
                                z[e] = a.interleaved ? __byte_perm(x[e], 0, 0x1032) : __shfl_sync(0xffffffffu, x[e], partner);
                            if (turned) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 y = __ffma2_rn(make_float2(bf16_lo(z[e]), bf16_hi(z[e])), si[e],
                                                                __fmul2_rn(make_float2(bf16_lo(x[e]), bf16_hi(x[e])), co[e]));
                                    x[e] = pack_bf16x2(y.x, y.y);
                                }
                            }
                        }
                        if (head < HG) *reinterpret_cast<uint4*>(dst + head * kHeadDim) = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
            }
            // the next row's first loads, before this row's other heads
            const uint4 now = ov;
            if (i + teams < rows) {
                if (member < tq) load_q(i + teams, member, w);
                if (other0 < others) ov = load_other(i + teams, other0);
            }
            if (r < 0) continue;
            // ---- key, value and index heads
#pragma unroll 1
            for (int t = other0; t < others; t += team) {
                int k, head, at;
                const bool there = other_task(t, k, head, at), index = k >= 3;
                const uint4 v = t == other0 ? now : load_other(i, t);
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                const int dim = k == 2 ? 0 : (index ? a.rope_index_dim : a.rope_dim), half = dim / 2;
                const bool turned = at < dim, lower = at < half;
                const int partner = turned && !a.interleaved ? lane + (lower ? dim / 16 : -(dim / 16)) : lane;
                const float2* cs = &turn[i][(index ? kHeadDim / 2 : 0) + (a.interleaved ? at / 2 : (lower ? at : at - half))];
                float y[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t z = a.interleaved ? __byte_perm(x[e], 0, 0x1032) : __shfl_sync(0xffffffffu, x[e], partner);
                    y[2 * e] = bf16_lo(x[e]);
                    y[2 * e + 1] = bf16_hi(x[e]);
                    if (turned) {
                        const float2 t0 = cs[a.interleaved ? e : 2 * e], t1 = cs[a.interleaved ? e : 2 * e + 1];
                        const float s0 = lower || a.interleaved ? -t0.y : t0.y, s1 = lower && !a.interleaved ? -t1.y : t1.y;
                        y[2 * e] = fmaf(bf16_lo(z), s0, y[2 * e] * t0.x);
                        y[2 * e + 1] = fmaf(bf16_hi(z), s1, y[2 * e + 1] * t1.x);
                    }
                }
                if (a.kv_int8 && !index) {  // the 16 lanes of a key or value head
                    uint32_t top = 0;  // largest magnitude as bits: a NaN counts as larger than infinity
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (there && row.cache >= 0) {
                        const float scale = __fdiv_rn(__uint_as_float(top), 127.f);
                        uint2 code = make_uint2(0u, 0u);
                        if (scale > 0.f && scale < INFINITY) code = ap_codes(y, scale);
                        const int64_t o = row.cache * H + head;
                        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(k == 1 ? a.k_cache : a.v_cache) + o * kHeadDim + at) = code;
                        if (at == 0) (k == 1 ? a.k_scale : a.v_scale)[o] = scale;
                    }
                } else if (kCodes && k == 4) {  // the 8 lanes of an index head
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    bool near = false;
                    if (there && row.cache >= 0) {
                        const int e = ap_index_exp(top);
                        const int64_t o = row.cache * a.KH + head;
                        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.ik_cache) + o * kIndexDim + at) =
                            e == -128 ? make_uint2(0u, 0u) : ap_index_codes(y, e);
                        if (at == 0) a.ik_exp[o] = static_cast<int8_t>(e);
                        // A value so near to a half, or a maximum to where the exponent changes, that the fp32 rotation may be on
                        // its other side (an angle and its cosine off by 2.2e-7, two roundings, 254 steps at most: 9e-5 of one).
                        // So may a head that is not finite in 32 bits: two values near 3.4e38 are turned past them.
                        near = turned && e == -128;
                        if (turned && e != -128) {
                            const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23), most = __uint_as_float(top) * f;
                            near = fabsf(most - 127.f) < kApNear || fabsf(most - 63.5f) < kApNear;
#pragma unroll
                            for (int c = 0; c < 8; ++c) near |= fabsf(y[c] * f - rintf(y[c] * f)) > 0.5f - kApNear;
                        }
                    }
                    const uint32_t who = __ballot_sync(0xffffffffu, near);
                    if (at == 0 && (who >> lane & 0xffu)) again_of[atomicAdd(&again, 1)] = static_cast<uint16_t>(8 * i + head);
                } else if (there && (k == 3 || row.cache >= 0)) {
                    uint16_t* dst = k == 3 ? a.iq_out + (r * H + head) * kIndexDim
                                  : k == 4 ? static_cast<uint16_t*>(a.ik_cache) + (row.cache * a.KH + head) * kIndexDim
                                           : static_cast<uint16_t*>(k == 1 ? a.k_cache : a.v_cache) + (row.cache * H + head) * kHeadDim;
                    *reinterpret_cast<uint4*>(dst + at) =
                        turned ? make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                            pack_bf16x2(y[6], y[7]))
                               : v;
                }
                __syncwarp();
            }
        }
        if constexpr (kCodes) {
            __syncthreads();
            for (int w = warp; w < again; w += kApWarps) ap_index_again(a, row_of[again_of[w] >> 3], again_of[w] & 7, lane);
        }
    }
    // Few rows: CTA 0 looks at every row once more and stores the word, so that no kernel has to clear it first.
    if (check_all) {
        if (blockIdx.x != 0) return;
        __syncthreads();
        if (tid < a.total_rows && gridDim.x > 1) {
            ApRow x{-1, 0, -1};
            const uint32_t bad = ap_find(a, tid, x);
            if (bad) atomicOr(&err, bad);
        }
        __syncthreads();
        if (tid == 0) *a.err = err;
    } else {
        __syncthreads();
        if (tid == 0 && err) atomicOr(a.err, err);
    }
}

cudaError_t run_append_cache(const AppendArgs& a, cudaStream_t stream) {
    if (a.total_rows > kApCheckRows) {
        cudaError_t e = cudaMemsetAsync(a.err, 0, sizeof(uint32_t), stream);
        if (e != cudaSuccess) return e;
    }
    // one CTA for each of the GPU's places (three an SM), as many rows as that makes (few rows: one a CTA)
    const int64_t places = 3 * static_cast<int64_t>(device_sm_count());
    const int64_t share = (static_cast<int64_t>(a.total_rows) + places - 1) / places;
    const int rows = static_cast<int>(share > kApRows ? kApRows : share);
    const int64_t need = (static_cast<int64_t>(a.total_rows) + rows - 1) / rows, cap = places;
    // warps that share a row (4,096 rows of 4 x 16 heads: 55, 49, 47 and 45 us with 1, 2, 4 and 8; 2,300 rows of 8 x 5: 31, 31, 29, 31)
    const int team = rows > 1 ? 4 : kApWarps;
    auto* kernel = a.ik_exp ? append_cache_kernel<true> : append_cache_kernel<false>;
    kernel<<<static_cast<unsigned>(need < cap ? need : cap), kApThreads, 0, stream>>>(a, rows, team);
    return cudaGetLastError();
}

}  // namespace msa
