// Attention over every cached position, decode family (1 to 8 rows a sequence).
//   out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m),  x_t = scale log2(e) q.k_t,  m = max_t x_t
// in one pass: a running maximum m, sum l and unnormalised output O per (row, query head), rescaled by
// 2^(m - m') when the maximum grows, and the parts of a sequence that several CTAs walk joined by the same rule.
//
// Bound by memory: each cached position is H x 512 bytes (264 with an int8 cache) that are read once for 16 (row, query
// head) pairs (more: bf16 windows are the window kernel's; int8 windows read the cache once for every 16).  The cache is split over its length: one CTA per SM takes an even share of all
// 64-position blocks of all sequences (from the lengths on the device, so ragged batches balance) and streams them
// through a ring of shared-memory stages, one (block, KV head) tile of K and V each, by TMA boxes issued by two
// producer warps.  Heads of a block are neighbours in the ring, so memory is read in whole 64 H-row runs.  Eight
// consumer warps take the tiles in turn; 8 is a multiple of H, so a warp stays with one head and keeps its queries (A
// operand, 16 (row, head) pairs) and O (accumulators) in registers.  S = Q K^T and O += P V run on mma.sync
// m16n8k16: 16 rows are all a tile has (tcgen05 wants 128), and 12 to 16 FLOP a byte are well within its rate.
//
// P enters the second product as two bf16 parts (2^-16 of a weight; bf16 outputs) or three (2^-24; fp32 outputs),
// taken from the accumulators of the first as they lie.
//
// int8 caches: the tiles are widened in registers to f16, exactly, by 1.25 instructions a value (bf16, whose 8 bits
// cannot hold the bias that such a conversion adds, takes 2): byte b, its sign bit flipped, under the exponent of
// 1024 is 1152 + b.  The order of the dimensions inside a dot product is free, so a lane takes 16-byte runs of its
// keys, and the second product's pairs of keys come from transposed loads of byte pairs.  Queries become f16 times a
// power of two for each row (its largest value in [2^8, 2^9): bf16's 8 bits fit; what lies 2^-22 below the row's
// largest loses bits).  The key scale multiplies the score and the value scale the weight.  A weight is 2^14 2^(x - m)
// times the value scale over a power of two not below any of the scales so far, in one f16 part (2^-11; bf16
// outputs) or two (2^-22; fp32): at most 2^14.  A tile with a scale below 2^-14 of that power of two (one far larger may
// be a drafted token's that earlier rows do not see) is summed key by key in fp32 instead, nine times slower (377 us
// where all tiles of the 43 us below are such, 68 us where one of 50 is).
//
// Where a sequence begins and ends inside one CTA, the CTA writes its output; else each CTA leaves its part (O, m,
// l) in the workspace, at most two a CTA, and dense_combine_kernel joins them.
//
// Measured (with the combine): 4 rows at 65,536, 4 x 16 heads, 92 us called back to back, 95 as a graph of one call
// (whose start nothing overlaps), 7.08 TB/s while every SM streams (they end 77 to 86 us in, the combine 4 us later); 8
// int8 sequences of 1,024 to 196,608, 43 and 46 us, bound by the 1,730 instructions a tile and warp, two warps a scheduler
// (42 % of the issue slots taken, waits on the instruction before the rest; registers leave no room for a third); 64
// sequences of 3 to 4,096, 8 x 4 heads, 37 and 40 us, a third of it before the first tile and after the last.
#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace msa {

constexpr int kDdConsumers = 8;
// Two warpgroups of consumers and one whose first two warps are the producers.  Registers move from the last to the others:
// launched with 168 a thread (64,512), 256 x 208 + 128 x 88 = 64,512 after the split.
constexpr int kDdThreads = 384;
constexpr int kDdMergeWords = 32 + 4;  // half of O, m and l of a lane
constexpr int kDdPrefix = 256;         // sequences whose prefixes are kept in shared memory (more: in the workspace)

// Tile i lands in stage i % kStages and completes barrier i % 16.  16 is a multiple of the consumers, so each of them
// sees its barriers' phases one after the other (a warp that saw only some of a stage's phases could not tell them
// apart by their parity), and with at most 16 stages no barrier is armed again before its last phase was seen.
constexpr int kDdFull = 16;

template <bool kInt8>
struct DdCfg {
    static constexpr int kPlane = kInt8 ? kBlock * kHeadDim : kBlock * kHeadDim * 2;  // K or V of a tile
    static constexpr int kStageBytes = 2 * kPlane + (kInt8 ? 1024 : 0);               // int8: 64 key, 64 value scales
    static constexpr int kStages = kInt8 ? 12 : 6;  // even: see the producers
    static constexpr int kMergeBytes = 4 * kDdMergeWords * 32 * 4;
    static_assert(kStages <= kDdFull, "a tile's barrier must not be armed twice ahead of its consumer");
    static constexpr int kBarArrivals = kInt8 ? 33 : 1;  // the producer lane, and the scale copies of the 32 lanes
};

__device__ __forceinline__ void dd_ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void dd_ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void dd_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float dd_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 dd_lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void dd_mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Bytes 0 and 2 of w (signed) as two f16: with the sign bit flipped and the exponent of 1024 above it a byte b reads
// as 1152 + b, exactly.
__device__ __forceinline__ uint32_t dd_even_f16(uint32_t w) {
    const uint32_t u = (w & 0x00FF00FFu) ^ 0x64806480u, bias = 0x64806480u;
    __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&bias));
    return *reinterpret_cast<uint32_t*>(&r);
}
// The same without taking the 1152 off.
__device__ __forceinline__ uint32_t dd_even_biased(uint32_t w) { return (w & 0x00FF00FFu) ^ 0x64806480u; }
__device__ __forceinline__ uint32_t dd_pack_f16(float lo, float hi) {
    __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ void dd_sync_consumers() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// A sequence's place in the work: its blocks, tiles of 16 (row, head) pairs, and what its rows need.
struct DdSeq {
    int b, c0, n, L, blocks, tiles;
};

__device__ __forceinline__ int dd_blocks(int L) { return (L + kBlock - 1) / kBlock; }

// Units (blocks x tiles) and tiles of sequence b; 0 if it is not of the decode family or its metadata is bad.
__device__ __forceinline__ int dd_units(const DenseArgs& a, int b, int& tiles, bool& bad) {
    bad = false;
    tiles = 0;
    const int c0 = a.cu_rows[b], n = a.cu_rows[b + 1] - c0, L = a.cache_lens[b];
    const bool placed = seq_rows_ok(a.cache, b, L, a.cache_tokens);  // (loads that need not wait for one another)
    if (n == 0 || n > kDecodeMaxRows || n * a.G > a.window_above) return 0;
    if (n < 0 || n > a.max_rows_per_seq || c0 < 0 || c0 + n > a.total_rows || L < n || L > a.max_cache_len || !placed) {
        bad = true;
        return 0;
    }
    tiles = (n * a.G + 15) / 16;
    return dd_blocks(L) * tiles;
}

__device__ __forceinline__ DdSeq dd_seq(const DenseArgs& a, int b) {
    DdSeq s;
    s.b = b;
    s.c0 = a.cu_rows[b];
    s.n = a.cu_rows[b + 1] - s.c0;
    s.L = a.cache_lens[b];
    s.blocks = dd_blocks(s.L);
    s.tiles = (s.n * a.G + 15) / 16;
    return s;
}

// CTAs that take a share of the tiles (unit u, head h: tile u H + h).  Going on to another segment (a sequence's 16 pairs)
// holds a CTA's warps up as some tiles would, so a segment counts for that many more: the shares divide evenly the line
// of all tiles with dd_extra of nothing before the first of each segment, from the very first tile on.  (With even tiles,
// of the shares of 64 short sequences those with four segments ended 10 us after those with one, 29 of 44 us, and the
// two-segment shares of 8 ragged int8 sequences 5 us after the others, 34 of 50.)
__device__ __forceinline__ int dd_shares(int64_t total, int grid) { return static_cast<int>(min(total, static_cast<int64_t>(grid))); }
__device__ __forceinline__ int dd_extra(bool int8) { return int8 ? 16 : 4; }
// Where share c begins.
__device__ __forceinline__ int64_t dd_cut(int64_t line, int extra, int c, int shares) {
    const int64_t n = line - extra;
    if (n * shares < (int64_t{1} << 32)) return extra + static_cast<uint32_t>(n) * static_cast<uint32_t>(c) / static_cast<uint32_t>(shares);
    return extra + n * c / shares;
}

__device__ __forceinline__ int dd_div(int64_t x, int64_t y) {
    if (((x | y) >> 32) == 0) return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
    return static_cast<int>(x / y);
}

// The tile at position `at` of that line (`extra` is where the next segment begins); b: its sequence, or one before it
// that has none.
__device__ __forceinline__ int64_t dd_tile_at(const int32_t* units, const int32_t* segs, int num_seqs, int H, int extra, int64_t at, int& b) {
    int lo = 0, hi = num_seqs;  // largest b that begins at or before it
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int64_t>(units[mid]) * H + static_cast<int64_t>(segs[mid]) * extra <= at) lo = mid; else hi = mid;
    }
    b = lo;
    const int u = units[lo], n = segs[lo + 1] - segs[lo];
    if (n == 0) return static_cast<int64_t>(u) * H;
    const int all = units[lo + 1] - u, blocks = n == 1 ? all : all / n, per = blocks * H + extra;
    const int off = static_cast<int>(at - static_cast<int64_t>(u) * H - static_cast<int64_t>(segs[lo]) * extra);
    const int mt = off < per ? 0 : off / per;
    return static_cast<int64_t>(u + mt * blocks) * H + max(0, off - mt * per - extra);
}

// Writes two neighbouring outputs of (row, head) pair m of a sequence, heads of KV head h.
__device__ __forceinline__ void dd_store2(const DenseArgs& a, const DdSeq& s, int h, int m, int d, float x, float y) {
    const int i = m / a.G, g = m - i * a.G;
    const int64_t o = ((static_cast<int64_t>(s.c0 + i) * a.H + h) * a.G + g) * kHeadDim + d;
    if (a.out_bf16)
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + o) = pack_bf16x2(x, y);
    else
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + o) = make_float2(x, y);
}

// int8 tiles whose value scales reach below this part of the largest so far (or of a later token's, which rows before it
// must not notice): f16 weights would have too few bits, so their keys are added one by one.
constexpr float kDdApart = 6.103515625e-05f;  // 2^-14

// O += weights x values of the keys of an int8 tile up to `last`, in fp32.  The weights lie over the stage's keys, [16][64];
// o: the lane's 16 x 4 accumulators, in units of 1 / vinv; pos: its rows' positions in the block.
template <int kPlane>
static __device__ __noinline__ void dd_add_by_key(uint8_t* stage, int last, int2 pos, float* o, float vinv) {
    const float* weights = reinterpret_cast<const float*>(stage);
    const float* scales = reinterpret_cast<const float*>(stage + 2 * kPlane + 256);
    const int lane = threadIdx.x & 31, grp = lane >> 2, tig = lane & 3;
    const float* w0 = weights + grp * kBlock;
    const float* w1 = w0 + 8 * kBlock;
    for (int chunk = 0; chunk < 8; ++chunk) {  // (dims as the lane's columns have them)
        float* y = o + 8 * chunk;
        float a[8] = {y[0], y[4], y[1], y[5], y[2], y[6], y[3], y[7]};
#pragma unroll 4
        for (int key = 0; key < last; ++key) {
            const char4 x = *reinterpret_cast<const char4*>(stage + kPlane + key * 128 + ((chunk ^ (key & 7)) << 4) + 4 * tig);
            const float v = scales[key] * vinv, f0 = w0[key] * v, f1 = w1[key] * v;
            if (key <= pos.x) {
                a[0] = fmaf(f0, x.x, a[0]);
                a[1] = fmaf(f0, x.y, a[1]);
                a[2] = fmaf(f0, x.z, a[2]);
                a[3] = fmaf(f0, x.w, a[3]);
            }
            if (key <= pos.y) {
                a[4] = fmaf(f1, x.x, a[4]);
                a[5] = fmaf(f1, x.y, a[5]);
                a[6] = fmaf(f1, x.z, a[6]);
                a[7] = fmaf(f1, x.w, a[7]);
            }
        }
        y[0] = a[0], y[4] = a[1], y[1] = a[2], y[5] = a[3];
        y[2] = a[4], y[6] = a[5], y[3] = a[6], y[7] = a[7];
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the stage's next copy
}

// t += what was set aside, in t's units.  Both: the lane's 16 x 4 accumulators, the maxima of its two rows and the power
// of two that the value scales are divided by, none of which fall.
constexpr int kDdAside = 512;  // tiles of a warp: 2,048 additions, 1.2e-4
static __device__ __noinline__ void dd_join_aside(const float* aside, float* t, bool some) {
    if (!some) return;
    const float unit = t[66] > 0.f ? aside[66] / t[66] : 1.f;
    for (int e = 0; e < 2; ++e) {
        const float f = aside[64 + e] == -INFINITY ? 0.f : dd_exp2(aside[64 + e] - t[64 + e]) * unit;
        for (int x = 2 * e; x < 64; x += 4) {
            t[x] = fmaf(aside[x], f, t[x]);
            t[x + 1] = fmaf(aside[x + 1], f, t[x + 1]);
        }
    }
}

template <int H, bool kInt8, int kParts>
__global__ void __launch_bounds__(kDdThreads, 1) dense_decode_kernel(const __grid_constant__ CUtensorMap k_map,
                                                                    const __grid_constant__ CUtensorMap v_map,
                                                                    const DenseArgs a) {
    using Cfg = DdCfg<kInt8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* merge = reinterpret_cast<float*>(ring + Cfg::kStages * Cfg::kStageBytes);
    // [num_seqs + 1]; in the workspace every CTA writes the same values
    int32_t* prefix = a.num_seqs < kDdPrefix ? reinterpret_cast<int32_t*>(ring + Cfg::kStages * Cfg::kStageBytes + Cfg::kMergeBytes)
                                             : a.unit_prefix;
    int32_t* segs = prefix + (a.num_seqs < kDdPrefix ? kDdPrefix : a.num_seqs + 1);  // the same of segments
    __shared__ uint64_t full[kDdFull], empty[Cfg::kStages];
    __shared__ int2 warp_tot[kDdThreads / 32];
    __shared__ uint32_t err;
    constexpr int kTailWarps = kInt8 ? 1 : kDdConsumers;  // (bf16 caches alone need it)
    __shared__ float tail_w[kTailWarps][16][kDecodeMaxRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < kDdFull; ++s) mbar_init(&full[s], Cfg::kBarArrivals);
        for (int s = 0; s < Cfg::kStages; ++s) mbar_init(&empty[s], 1);
        fence_mbar_init();
        err = 0;
        prefetch_tmap(&k_map);
        prefetch_tmap(&v_map);
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- exclusive prefixes of the sequences' units and segments (a block-wide scan, kDdThreads sequences at a time)
    int2 carry = make_int2(0, 0);
    for (int base = 0; base < a.num_seqs; base += kDdThreads) {
        const int b = base + tid;
        bool bad = false;
        int2 mine = make_int2(0, 0);
        if (b < a.num_seqs) mine.x = dd_units(a, b, mine.y, bad);
        if (bad && blockIdx.x == 0) atomicOr(&err, kErrBadMetadata);
        int2 incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl.x, o), w = __shfl_up_sync(0xffffffffu, incl.y, o);
            if (lane >= o) incl = make_int2(incl.x + v, incl.y + w);
        }
        if (lane == 31) warp_tot[warp] = incl;
        __syncthreads();
        int2 before = make_int2(0, 0), total = make_int2(0, 0);
        for (int w = 0; w < kDdThreads / 32; ++w) {
            const int2 t = warp_tot[w];
            if (w < warp) before = make_int2(before.x + t.x, before.y + t.y);
            total = make_int2(total.x + t.x, total.y + t.y);
        }
        if (b < a.num_seqs) {
            prefix[b] = carry.x + before.x + incl.x - mine.x;
            segs[b] = carry.y + before.y + incl.y - mine.y;
        }
        __syncthreads();
        carry = make_int2(carry.x + total.x, carry.y + total.y);
    }
    if (tid == 0) {
        prefix[a.num_seqs] = carry.x;
        segs[a.num_seqs] = carry.y;
    }
    __syncthreads();
    if (blockIdx.x == 0 && a.num_seqs < kDdPrefix)
        for (int b = tid; b <= a.num_seqs; b += kDdThreads) {
            a.unit_prefix[b] = prefix[b];
            a.unit_prefix[a.num_seqs + 1 + b] = segs[b];
        }
    // this CTA's tiles: [begin, begin + n) of all; the first is head h_off of unit u0
    const int64_t total = static_cast<int64_t>(carry.x) * H, line = total + static_cast<int64_t>(carry.y) * dd_extra(kInt8);
    const int shares = dd_shares(total, gridDim.x);  // CTAs with work (some of them none, where segments are very short)
    const bool idle = static_cast<int>(blockIdx.x) >= shares;
    int first_b = 0, n_tiles = 0;
    int64_t begin = 0;
    if (!idle) {  // even lanes find where it begins, odd ones where it ends
        int b;
        const int64_t at = dd_tile_at(prefix, segs, a.num_seqs, H, dd_extra(kInt8),
                                      dd_cut(line, dd_extra(kInt8), blockIdx.x + (lane & 1), shares), b);
        first_b = __shfl_sync(0xffffffffu, b, 0);
        begin = __shfl_sync(0xffffffffu, at, 0);
        n_tiles = static_cast<int>(__shfl_sync(0xffffffffu, at, 1) - begin);
    }
    const int u0 = static_cast<int>(begin / H), h_off = static_cast<int>(begin % H);
    const int u1 = n_tiles == 0 ? u0 : u0 + (h_off + n_tiles + H - 1) / H;

    if (warp >= kDdConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp < kDdConsumers + 2) {
        // ---------------- two producers, the even and the odd tiles (one warp's barrier tests, copies and scale copies,
        // 870 cycles an int8 tile, held 8 ragged int8 sequences to 59 us).  With an even number of stages each of them
        // sees every phase of its stages.  32 blocks' cache rows at a time, one lane each, then their tiles in order.
        static_assert(Cfg::kStages % 2 == 0, "a producer must see every phase of its stages");
        const int odd = warp - kDdConsumers;
        int sent = 0;  // the CTA's tiles up to this warp's last copy
        int b = first_b;
        bool alive = true;
        for (int base = u0; base < u1 && alive; base += 32) {
            const int u = base + lane;
            int64_t row = -1;
            int live = 0;
            if (u < u1) {
                while (u >= prefix[b + 1]) ++b;
                const int L = a.cache_lens[b], blocks = dd_blocks(L);
                const int j = (u - prefix[b]) % blocks;
                live = min(kBlock, L - j * kBlock);
                row = block_row(a.cache, b, static_cast<int64_t>(j) * kBlock);
                if (row < 0) {  // page outside the pool: nothing of it is read (a box past the cache is zeros)
                    atomicOr(&err, kErrBadMetadata);
                    row = a.cache_tokens;
                    live = 0;
                }
            }
            const int count = min(32, u1 - base);
            for (int i = 0; i < count && alive; ++i) {
                const int64_t r = __shfl_sync(0xffffffffu, row, i);
                const int n = __shfl_sync(0xffffffffu, live, i);
#pragma unroll 1
                for (int h = 0; h < H; ++h) {
                    const int tile = (base - u0 + i) * H + h - h_off;  // of the CTA's
                    if (tile < 0 || tile >= n_tiles || (tile & 1) != odd) continue;
                    const int s = tile % Cfg::kStages;
                    int ok = 1;
                    if (lane == 0 && tile >= Cfg::kStages) ok = mbar_wait(&empty[s], ((tile / Cfg::kStages) - 1) & 1, &err);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) {
                        alive = false;
                        break;
                    }
                    uint8_t* st = ring + s * Cfg::kStageBytes;
                    uint64_t* bar = &full[tile % kDdFull];
                    sent = tile + 1;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, 2 * Cfg::kPlane);
                        if constexpr (kInt8) {
                            tma_load_3d(st, &k_map, bar, 0, h, static_cast<int>(r));
                            tma_load_3d(st + Cfg::kPlane, &v_map, bar, 0, h, static_cast<int>(r));
                        } else {
#pragma unroll
                            for (int half = 0; half < 2; ++half)
                                tma_load_3d(st + half * (Cfg::kPlane / 2), &k_map, bar, 64 * half, h, static_cast<int>(r));
#pragma unroll
                            for (int half = 0; half < 2; ++half)
                                tma_load_3d(st + Cfg::kPlane + half * (Cfg::kPlane / 2), &v_map, bar, 64 * half, h,
                                            static_cast<int>(r));
                        }
                    }
                    if constexpr (kInt8) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {  // 64 key scales, 64 value scales; those past the length are not read
                            const int key = (c & 1) * 32 + lane;
                            const float* src = (c < 2 ? a.k_scale : a.v_scale) + (r + key) * H + h;
                            const uint32_t dst = smem_u32(st + 2 * Cfg::kPlane + (c >> 1) * 256 + key * 4);
                            if (key < n) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
                        }
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
                    }
                }
            }
        }
        // no copy of this warp may be in flight when the CTA ends
        if (lane == 0)
            for (int s = odd; s < kDdFull && s < sent; s += 2) mbar_wait(&full[s], ((sent - 1 - s) / kDdFull) & 1, &err);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---------------- consumer warp: every 8th tile, all of head warp % H
        const int grp = lane >> 2, tig = lane & 3, h = warp % H;
        // int8, bf16 outputs: the keys keep their bias and the accumulators begin at -1152 sum q (its cancellation costs
        // some 1e-5 of a score's spread, far below the outputs' rounding; fp32 outputs take the bias off)
        constexpr bool kBiased = kInt8 && kParts == 1, kAside = kInt8 && kParts == 1;
        bool alive = true;
        int i = (warp - static_cast<int>(begin % kDdConsumers)) & (kDdConsumers - 1), b = first_b;
        for (int cur = 0; cur < n_tiles;) {
            const int u = u0 + (cur + h_off) / H;
            while (u >= prefix[b + 1]) ++b;
            const DdSeq s = dd_seq(a, b);
            const int mt = (u - prefix[b]) / s.blocks, seg0 = prefix[b] + mt * s.blocks, seg1 = seg0 + s.blocks;
            // this CTA's part of the (sequence, 16 pairs): its tiles [cur, end)
            const int seg_first = (seg0 - u0) * H - h_off, seg_last = (seg1 - u0) * H - h_off, end = min(n_tiles, seg_last);
            const int pairs = min(16, s.n * a.G - 16 * mt);
            // rows grp and grp + 8 of the tile: (row, head) pair, position, whether it exists
            int pos[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) pos[e] = s.L - s.n + min(16 * mt + grp + 8 * e, s.n * a.G - 1) / a.G;
            const int first_pos = s.L - s.n + 16 * mt / a.G;  // the tile's earliest row
            uint32_t qa[8][4];
            float qf[2];  // factor from the product to the log2 domain, rows grp and grp + 8
            float qsum[2] = {0.f, 0.f};  // int8, biased keys: what the bias adds to the rows' products, negated
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int m = 16 * mt + min(grp + 8 * e, pairs - 1), qi = m / a.G, g = m - qi * a.G;
                const uint32_t* src = reinterpret_cast<const uint32_t*>(
                    a.q + ((static_cast<int64_t>(s.c0 + qi) * H + h) * a.G + g) * kHeadDim);
                qf[e] = a.scale_log2;
                if constexpr (kInt8) {
                    // dims 32 tig + 4 ks + {0, 2} and {1, 3}: the order in which a word of four key bytes is widened
                    float v[32], top = 0.f;
#pragma unroll
                    for (int x4 = 0; x4 < 4; ++x4) {
                        const uint4 w4 = *reinterpret_cast<const uint4*>(src + 16 * tig + 4 * x4);
                        const uint32_t ws[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int x = 4 * x4 + y;
                            v[2 * x] = bf16_lo(ws[y]);
                            v[2 * x + 1] = bf16_hi(ws[y]);
                            top = fmaxf(top, fmaxf(fabsf(v[2 * x]), fabsf(v[2 * x + 1])));
                        }
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const uint32_t ex = min(max(__float_as_uint(top) >> 23, 9u), 253u);
                    const float f = __uint_as_float((262u - ex) << 23);  // 2^(8 - exponent of the row's largest)
                    qf[e] *= __uint_as_float((ex - 8u) << 23);
                    float all = 0.f;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        qa[ks][e] = dd_pack_f16(v[4 * ks] * f, v[4 * ks + 2] * f);
                        qa[ks][2 + e] = dd_pack_f16(v[4 * ks + 1] * f, v[4 * ks + 3] * f);
                        const float2 q02 = __half22float2(*reinterpret_cast<const __half2*>(&qa[ks][e]));
                        const float2 q13 = __half22float2(*reinterpret_cast<const __half2*>(&qa[ks][2 + e]));
                        all += (q02.x + q02.y) + (q13.x + q13.y);
                    }
                    all += __shfl_xor_sync(0xffffffffu, all, 1);
                    all += __shfl_xor_sync(0xffffffffu, all, 2);
                    qsum[e] = kBiased ? -1152.f * all : 0.f;
                } else {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {  // dims 16 ks + 2 tig, + 8
                        qa[ks][e] = src[8 * ks + tig];
                        qa[ks][2 + e] = src[8 * ks + 4 + tig];
                    }
                }
            }
            float vref = 0.f, vinv = 0.f;  // int8: the power of two that the value scales are divided by, its inverse
            float o[16][4], mrun[2] = {-INFINITY, -INFINITY}, lrun[2] = {0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < 16; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
            float aside[kAside ? 67 : 1];  // O, maxima and unit of the tiles before (in local memory)
            int since = 0;                  // tiles since
            bool some = false;              // whether there were any

            for (; i < end; i += kDdConsumers) {
                if constexpr (kAside) {
                    if (since++ == kDdAside) {
                        float t[67];
#pragma unroll
                        for (int x = 0; x < 64; ++x) t[x] = o[x >> 2][x & 3];
                        t[64] = mrun[0];
                        t[65] = mrun[1];
                        t[66] = vref;
                        dd_join_aside(aside, t, some);
#pragma unroll
                        for (int x = 0; x < 64; ++x) {
                            aside[x] = t[x];
                            o[x >> 2][x & 3] = 0.f;
                        }
                        aside[64] = mrun[0];
                        aside[65] = mrun[1];
                        aside[66] = vref;
                        some = true;
                        since = 1;
                    }
                }
                const int st = i % Cfg::kStages, j = u0 + (i + h_off) / H - seg0, t0 = j * kBlock;
                if (alive) alive = mbar_wait(&full[i % kDdFull], (i / kDdFull) & 1, &err);
                if (!alive) continue;
                uint8_t* stage = ring + st * Cfg::kStageBytes;
                const uint32_t kb = smem_u32(stage), vb = kb + Cfg::kPlane;
                const bool edge = t0 + kBlock > first_pos + 1;  // some key is hidden from some row
                float c[8][4];
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) {
                    c[nt][0] = c[nt][1] = qsum[0];
                    c[nt][2] = c[nt][3] = qsum[1];
                    if constexpr (kInt8) {
                        const int row = nt * 8 + grp;
                        const uint4 w0 = dd_lds128(kb + row * 128 + (((2 * tig) ^ (row & 7)) << 4));
                        const uint4 w1 = dd_lds128(kb + row * 128 + (((2 * tig + 1) ^ (row & 7)) << 4));
                        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            if constexpr (kBiased) dd_mma_f16(c[nt], qa[ks], dd_even_biased(w[ks]), dd_even_biased(w[ks] >> 8));
                            else dd_mma_f16(c[nt], qa[ks], dd_even_f16(w[ks]), dd_even_f16(w[ks] >> 8));
                        }
                    } else {
                        const int row = nt * 8 + (lane & 7);
#pragma unroll
                        for (int k2 = 0; k2 < 4; ++k2) {  // 32 dims: chunks of 8 dims 4 (k2 & 1) .. + 3 of a half
                            uint32_t r[4];
                            const int chunk = (k2 & 1) * 4 + (lane >> 3);
                            dd_ldsm_x4(kb + (k2 >> 1) * (Cfg::kPlane / 2) + row * 128 + ((chunk ^ (row & 7)) << 4), r);
                            dd_mma(c[nt], qa[2 * k2], r[0], r[1]);
                            dd_mma(c[nt], qa[2 * k2 + 1], r[2], r[3]);
                        }
                    }
                }
                // int8: times the key scales; the value scales of the lane's 16 keys
                float2 vs[8];
                if constexpr (kInt8) {
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt) {
                        const float2 ks = *reinterpret_cast<const float2*>(stage + 2 * Cfg::kPlane + (nt * 8 + 2 * tig) * 4);
                        vs[nt] = *reinterpret_cast<const float2*>(stage + 2 * Cfg::kPlane + 256 + (nt * 8 + 2 * tig) * 4);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 x = __fmul2_rn(make_float2(c[nt][2 * e], c[nt][2 * e + 1]), ks);
                            c[nt][2 * e] = x.x;
                            c[nt][2 * e + 1] = x.y;
                        }
                    }
                }
                if (edge) {  // hidden keys -inf (scaled here: a scale of zero must not meet an infinity)
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt) {
                        const int t = t0 + nt * 8 + 2 * tig;
                        c[nt][0] = t > pos[0] ? -INFINITY : c[nt][0] * qf[0];
                        c[nt][1] = t + 1 > pos[0] ? -INFINITY : c[nt][1] * qf[0];
                        c[nt][2] = t > pos[1] ? -INFINITY : c[nt][2] * qf[1];
                        c[nt][3] = t + 1 > pos[1] ? -INFINITY : c[nt][3] * qf[1];
                        if constexpr (kInt8) {
                            if (t >= s.L) vs[nt].x = 0.f;
                            if (t + 1 >= s.L) vs[nt].y = 0.f;
                        }
                    }
                }
                const float f0 = edge ? 1.f : qf[0], f1 = edge ? 1.f : qf[1];  // what is left to multiply by
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) {
                    top[0] = fmaxf(top[0], fmaxf(c[nt][0], c[nt][1]));
                    top[1] = fmaxf(top[1], fmaxf(c[nt][2], c[nt][3]));
                }
                top[0] *= f0;
                top[1] *= f1;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                    top[e] = fmaxf(top[e], mrun[e]);
                }
                bool grew = top[0] > mrun[0] || top[1] > mrun[1], apart = false;
                float vnew = vref;
                if constexpr (kInt8) {
                    float big[8], low[8];
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt) {
                        big[nt] = fmaxf(fabsf(vs[nt].x), fabsf(vs[nt].y));
                        low[nt] = fminf(fabsf(vs[nt].x), fabsf(vs[nt].y));
                    }
#pragma unroll
                    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
                        for (int nt = 0; nt < d; ++nt) {
                            big[nt] = fmaxf(big[nt], big[nt + d]);
                            low[nt] = fminf(low[nt], low[nt + d]);
                        }
                    if (big[0] > vref && big[0] < INFINITY) {  // the next power of two, at most 2^127
                        vnew = __uint_as_float(min((__float_as_uint(big[0]) + 0x007FFFFFu) & 0x7F800000u, 0x7F000000u));
                        grew = true;
                    }
                    grew |= low[0] < vref * kDdApart;
                }
                if (__any_sync(0xffffffffu, grew)) {
                    if constexpr (kInt8) {  // the same in every lane
                        vnew = fmaxf(vnew, __shfl_xor_sync(0xffffffffu, vnew, 1));
                        vnew = fmaxf(vnew, __shfl_xor_sync(0xffffffffu, vnew, 2));
                        bool below = false;
#pragma unroll
                        for (int nt = 0; nt < 8; ++nt) {
                            below |= vs[nt].x != 0.f && fabsf(vs[nt].x) < vnew * kDdApart;
                            below |= vs[nt].y != 0.f && fabsf(vs[nt].y) < vnew * kDdApart;
                        }
                        apart = __any_sync(0xffffffffu, below);
                    }
                    const float fv = kInt8 ? (vnew > 0.f ? vref / vnew : 1.f) : 1.f;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = mrun[e] == -INFINITY ? 0.f : dd_exp2(mrun[e] - top[e]), fo = f * fv;
                        lrun[e] *= f;
                        mrun[e] = top[e];
#pragma unroll
                        for (int nt = 0; nt < 16; ++nt) {
                            o[nt][2 * e] *= fo;
                            o[nt][2 * e + 1] *= fo;
                        }
                    }
                    vref = vnew;
                    vinv = vnew > 0.f ? 1.f / vnew : 0.f;
                }
                constexpr float kLift = kInt8 ? 14.f : 0.f;  // f16 weights: 2^14 at most
                {
                    const float b0 = kLift - (mrun[0] == -INFINITY ? 0.f : mrun[0]), b1 = kLift - (mrun[1] == -INFINITY ? 0.f : mrun[1]);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float f = e ? f1 : f0, b = e ? b1 : b0;
                            float2 x = __ffma2_rn(make_float2(c[nt][2 * e], c[nt][2 * e + 1]), make_float2(f, f), make_float2(b, b));
                            x = make_float2(dd_exp2(x.x), dd_exp2(x.y));
                            sum[e] = __fadd2_rn(sum[e], x);
                            c[nt][2 * e] = x.x;
                            c[nt][2 * e + 1] = x.y;
                        }
                    lrun[0] += sum[0].x + sum[0].y;
                    lrun[1] += sum[1].x + sum[1].y;
                }
                if constexpr (kInt8) {
                    if (apart) {
                        float* weights = reinterpret_cast<float*>(stage);  // (the keys are done with)
                        float t[64];                                        // O goes through local memory here alone
#pragma unroll
                        for (int x = 0; x < 64; ++x) {
                            if (x < 32) weights[(grp + 8 * ((x & 3) >> 1)) * kBlock + (x >> 2) * 8 + 2 * tig + (x & 1)] = c[x >> 2][x & 3];
                            t[x] = o[x >> 2][x & 3];
                        }
                        __syncwarp();
                        dd_add_by_key<Cfg::kPlane>(stage, min(kBlock, s.L - t0), make_int2(pos[0] - t0, pos[1] - t0), t, vinv);
#pragma unroll
                        for (int x = 0; x < 64; ++x) o[x >> 2][x & 3] = t[x];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&empty[st]);
                        continue;
                    }
                    if (edge) {  // a hidden key's weight stays 0 whatever its scale is
#pragma unroll
                        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float v = (e & 1 ? vs[nt].y : vs[nt].x) * vinv;
                                c[nt][e] = c[nt][e] == 0.f ? 0.f : c[nt][e] * v;
                            }
                    } else {
#pragma unroll
                        for (int nt = 0; nt < 8; ++nt) {
                            const float2 v = __fmul2_rn(vs[nt], make_float2(vinv, vinv));
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float2 x = __fmul2_rn(make_float2(c[nt][2 * e], c[nt][2 * e + 1]), v);
                                c[nt][2 * e] = x.x;
                                c[nt][2 * e + 1] = x.y;
                            }
                        }
                    }
                } else if (edge) {
                    // Keys hidden from some row may hold anything: their values leave the products (zeroed in
                    // the stage) and those that later rows do see are added one by one below.
                    const int first = max(0, first_pos + 1 - t0);  // first such key of the block
                    const int last = min(kBlock, s.L - t0);         // keys from `last` on belong to no row
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = nt * 8 + 2 * tig + (e & 1);
                            if (key >= first) {
                                if (key < last) tail_w[warp % kTailWarps][grp + 8 * (e >> 1)][key - first] = c[nt][e];
                                c[nt][e] = 0.f;
                            }
                        }
                    __syncwarp();
                    for (int key = first; key < last; ++key) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (t0 + key > pos[e]) continue;
                            const float w = tail_w[warp % kTailWarps][grp + 8 * e][key - first];
#pragma unroll
                            for (int nt = 0; nt < 16; ++nt) {
                                const int chunk = nt & 7;
                                const uint32_t v2 = *reinterpret_cast<const uint32_t*>(
                                    stage + Cfg::kPlane + (nt >> 3) * (Cfg::kPlane / 2) + key * 128 +
                                    ((chunk ^ (key & 7)) << 4) + 4 * tig);
                                o[nt][2 * e] = fmaf(w, bf16_lo(v2), o[nt][2 * e]);
                                o[nt][2 * e + 1] = fmaf(w, bf16_hi(v2), o[nt][2 * e + 1]);
                            }
                        }
                    }
                    __syncwarp();
                    for (int x = first * 16 + lane; x < kBlock * 16; x += 32) {
                        const int key = x >> 4, chunk = x & 15;
                        *reinterpret_cast<uint4*>(stage + Cfg::kPlane + (chunk >> 3) * (Cfg::kPlane / 2) + key * 128 +
                                                  (((chunk & 7) ^ (key & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the stage's next copy
                    __syncwarp();
                }
                // O += P V, 16 keys a step.  The tensor cores cut what an addition loses instead of rounding it (a bias of
                // about 2^-24 each, 1.5e-4 after 33,280 keys), so a tile is summed by itself and then added to O; int8
                // caches with bf16 outputs, where that would cost 8 % (46.3 against 42.9 us for 8 ragged sequences), set
                // O aside every so many tiles instead.
                uint32_t pa[4][kParts][4];
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        float x = c[2 * kk + (f >> 1)][2 * (f & 1)], y = c[2 * kk + (f >> 1)][2 * (f & 1) + 1];
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            if constexpr (kInt8) {
                                pa[kk][part][f] = dd_pack_f16(x, y);
                                const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&pa[kk][part][f]));
                                x -= r.x;
                                y -= r.y;
                            } else {
                                pa[kk][part][f] = pack_bf16x2(x, y);
                                x -= bf16_lo(pa[kk][part][f]);
                                y -= bf16_hi(pa[kk][part][f]);
                            }
                        }
                    }
                constexpr bool kApart = !kAside;  // a tile's product by itself
                if constexpr (kInt8) {
#pragma unroll
                    for (int n4 = 0; n4 < 4; ++n4) {
                        // 32 dims: n-tile 2 x + y (x: 16-byte chunk 2 n4 + x, y: parity) has dim 16 chunk + 2 grp + y in column grp
                        float t[4][4];
#pragma unroll
                        for (int n = 0; n < 4; ++n) t[n][0] = t[n][1] = t[n][2] = t[n][3] = 0.f;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            // byte pairs (dims 2 grp, + 1) of keys 16 kk + 2 tig, + 1 and those 8 further, chunks 2 n4 and + 1
                            uint32_t r[4];
                            const int key = 16 * kk + ((lane >> 3) & 1) * 8 + (lane & 7), chunk = 2 * n4 + (lane >> 4);
                            dd_ldsm_x4_t(vb + key * 128 + ((chunk ^ (key & 7)) << 4), r);
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                const int sh = (n & 1) * 8, at = (n >> 1) * 2;
                                const uint32_t b0 = dd_even_f16(r[at] >> sh), b1 = dd_even_f16(r[at + 1] >> sh);
#pragma unroll
                                for (int part = 0; part < kParts; ++part)
                                    dd_mma_f16(kApart ? t[n] : o[4 * n4 + n], pa[kk][part], b0, b1);
                            }
                        }
                        if constexpr (kApart) {
#pragma unroll
                            for (int n = 0; n < 4; ++n)
#pragma unroll
                                for (int e = 0; e < 4; e += 2) {
                                    const float2 x = __fadd2_rn(make_float2(o[4 * n4 + n][e], o[4 * n4 + n][e + 1]), make_float2(t[n][e], t[n][e + 1]));
                                    o[4 * n4 + n][e] = x.x;
                                    o[4 * n4 + n][e + 1] = x.y;
                                }
                        }
                    }
                } else {
                    // 32 dims at a time, four accumulators in turn (each product waits for the last on its accumulator)
#pragma unroll
                    for (int n4 = 0; n4 < 4; ++n4) {
                        float t[4][4];
#pragma unroll
                        for (int n = 0; n < 4; ++n) t[n][0] = t[n][1] = t[n][2] = t[n][3] = 0.f;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            uint32_t r[2][4];
                            const int key = 16 * kk + (lane & 15);
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int n2 = 2 * n4 + y, chunk = (n2 & 3) * 2 + (lane >> 4);
                                dd_ldsm_x4_t(vb + (n2 >> 2) * (Cfg::kPlane / 2) + key * 128 + ((chunk ^ (key & 7)) << 4), r[y]);
                            }
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
#pragma unroll
                                for (int n = 0; n < 4; ++n)
                                    dd_mma(kApart ? t[n] : o[4 * n4 + n], pa[kk][part], r[n >> 1][2 * (n & 1)], r[n >> 1][2 * (n & 1) + 1]);
                        }
                        if constexpr (kApart) {
#pragma unroll
                            for (int n = 0; n < 4; ++n)
#pragma unroll
                                for (int e = 0; e < 4; e += 2) {
                                    const float2 x = __fadd2_rn(make_float2(o[4 * n4 + n][e], o[4 * n4 + n][e + 1]), make_float2(t[n][e], t[n][e + 1]));
                                    o[4 * n4 + n][e] = x.x;
                                    o[4 * n4 + n][e + 1] = x.y;
                                }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }

            if constexpr (kAside) {
                if (some) {
                    float t[67];
#pragma unroll
                    for (int x = 0; x < 64; ++x) t[x] = o[x >> 2][x & 3];
                    t[64] = mrun[0];
                    t[65] = mrun[1];
                    t[66] = vref;
                    dd_join_aside(aside, t, true);
#pragma unroll
                    for (int x = 0; x < 64; ++x) o[x >> 2][x & 3] = t[x];
                }
            }
            if constexpr (kInt8) {
#pragma unroll
                for (int nt = 0; nt < 16; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][e] *= vref;
            }
            // ---- the warps of a head join their parts (8 / H of them, by halves)
#pragma unroll
            for (int half = kDdConsumers / 2; half >= H; half >>= 1) {
                if ((begin + cur) % kDdConsumers == 0 && end - cur <= half) continue;  // warps from `half` on had no tile
                float f1[2], f2[2];
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // half of O at a time
                    dd_sync_consumers();
                    if (warp >= half && warp < 2 * half) {
                        float* dst = merge + (warp - half) * (kDdMergeWords * 32) + lane;
#pragma unroll
                        for (int x = 0; x < 32; ++x) dst[x * 32] = o[8 * part + (x >> 2)][x & 3];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            dst[(32 + e) * 32] = mrun[e];
                            dst[(34 + e) * 32] = lrun[e];
                        }
                    }
                    dd_sync_consumers();
                    if (warp < half) {
                        const float* src = merge + warp * (kDdMergeWords * 32) + lane;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (part == 0) {
                                const float m2 = src[(32 + e) * 32], m = fmaxf(mrun[e], m2);
                                f1[e] = mrun[e] == -INFINITY ? 0.f : dd_exp2(mrun[e] - m);
                                f2[e] = m2 == -INFINITY ? 0.f : dd_exp2(m2 - m);
                                mrun[e] = m;
                                lrun[e] = lrun[e] * f1[e] + src[(34 + e) * 32] * f2[e];
                            }
#pragma unroll
                            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                                for (int y = 0; y < 2; ++y)
                                    o[8 * part + nt][2 * e + y] =
                                        o[8 * part + nt][2 * e + y] * f1[e] + src[(nt * 4 + 2 * e + y) * 32] * f2[e];
                        }
                    }
                }
            }
            if (warp < H) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    lrun[e] += __shfl_xor_sync(0xffffffffu, lrun[e], 1);
                    lrun[e] += __shfl_xor_sync(0xffffffffu, lrun[e], 2);
                }
                const bool whole = cur == seg_first && end == seg_last;
                const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (cur == 0 ? 0 : 1)) * H + h;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int m = grp + 8 * e;
                    if (m >= pairs) continue;
                    float* part = a.part_o + (slot * 16 + m) * kHeadDim;
                    const float f = whole ? 1.f / lrun[e] : 1.f;
                    if (!whole && tig == 0)
                        *reinterpret_cast<float2*>(a.part_ml + (slot * 16 + m) * 2) = make_float2(mrun[e], lrun[e]);
#pragma unroll
                    for (int nt = 0; nt < 16; nt += 2) {
                        // two pairs of neighbouring dims.  bf16: columns 2 tig, + 1 of each n-tile; int8: the two n-tiles of a
                        // chunk have dims 16 chunk + 4 tig + {0, 2} and {1, 3} in the lane's columns
                        const float p0 = o[nt][2 * e] * f, p1 = (kInt8 ? o[nt + 1][2 * e] : o[nt][2 * e + 1]) * f;
                        const float p2 = (kInt8 ? o[nt][2 * e + 1] : o[nt + 1][2 * e]) * f, p3 = o[nt + 1][2 * e + 1] * f;
                        const int d0 = kInt8 ? 8 * nt + 4 * tig : 8 * nt + 2 * tig, d1 = kInt8 ? d0 + 2 : d0 + 8;
                        if (whole) {
                            dd_store2(a, s, h, 16 * mt + m, d0, p0, p1);
                            dd_store2(a, s, h, 16 * mt + m, d1, p2, p3);
                        } else {
                            *reinterpret_cast<float2*>(part + d0) = make_float2(p0, p1);
                            *reinterpret_cast<float2*>(part + d1) = make_float2(p2, p3);
                        }
                    }
                }
            }
            cur = end;
        }
    }
    __syncthreads();
    if (tid == 0) a.err_slots[blockIdx.x] = err;
}

// Joins the parts of the sequences that several CTAs walked.  CTA (x, h, z) takes a (sequence, tile), x itself where
// they are no more than the shares (by_tile: tiles a sequence may have), else the one in which boundary x + 1 of the
// shares is the first to fall, if any; of its (row, head) pairs every gridDim.z-th.  kShare warps share the parts of a
// pair, eight parts' loads in flight and 4 of the 128 values a lane: a running maximum m
// and sum of 2^(m_i - m) O_i in the parts' order within a warp, then over the warps: the same every time.  What bounds
// it is the chain of dependent loads (metadata, parts), so the metadata is read while the shares' CTAs still run.
template <int kThreads, int kShare>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) dense_combine_kernel(const DenseArgs a, int grid, int by_tile) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float4 sum_o[kWarps][32];
    __shared__ float2 sum_ml[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y, extra = dd_extra(a.kv_int8);
    // ---- which parts: from the inputs alone where a thread a sequence is enough (before the wait), else from the prefixes
    // that the shares' CTA 0 wrote
    int lo = by_tile > 0 ? blockIdx.x / by_tile : 0, mt = by_tile > 0 ? blockIdx.x % by_tile : 0;  // sequence, tile
    const bool early = by_tile > 0 && a.num_seqs <= kThreads;
    int begin = 0, units = 0, carry = 0;     // units before the sequence, of it, of all
    int seg_begin = 0, seg_carry = 0;        // segments before it, of all
    if (early) {
        __shared__ int sums[5][kWarps];
        bool bad;
        int tiles = 0;
        const int mine = tid < a.num_seqs ? dd_units(a, tid, tiles, bad) : 0;
        const int part[5] = {tid < lo ? mine : 0, tid == lo ? mine : 0, mine, tid < lo ? tiles : 0, tiles};
#pragma unroll
        for (int q = 0; q < 5; ++q) {
            const int sum = __reduce_add_sync(0xffffffffu, part[q]);
            if (lane == 0) sums[q][warp] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
            begin += sums[0][q];
            units += sums[1][q];
            carry += sums[2][q];
            seg_begin += sums[3][q];
            seg_carry += sums[4][q];
        }
    }
    DdSeq s{};
    int first = 0, last = 0, slot0 = 0;
    // the shares that hold its first and last tiles (the largest c that begins at or before the tile); the first share's part
    // is its second one unless the share began with it, the others' are the first of their shares
    auto find_parts = [&]() {
        const int64_t total = static_cast<int64_t>(carry) * a.H, line = total + static_cast<int64_t>(seg_carry) * extra;
        const int shares = dd_shares(total, grid), n_seg = s.blocks * a.H;  // the segment's tiles
        const int64_t at = static_cast<int64_t>(begin) * a.H + static_cast<int64_t>(seg_begin) * extra + static_cast<int64_t>(mt) * (n_seg + extra);
        first = dd_div((at + 1) * shares - 1, line - extra);
        last = dd_div((at + n_seg) * shares - 1, line - extra);
        slot0 = 2 * first + (dd_cut(line, extra, first, shares) < at ? 1 : 0);
    };
    if (early) {
        s = dd_seq(a, lo);
        if (units > 0 && mt < s.tiles) find_parts();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && h == 0 && blockIdx.z == 0 && warp == 0) {  // what the shares' CTAs found wrong
        uint32_t e = 0;
        for (int c = lane; c < grid; c += 32) e |= a.err_slots[c];
        e = __reduce_or_sync(0xffffffffu, e);
        if (lane == 0) {
            if (a.err_store) *a.err = e;
            else if (e) atomicOr(a.err, e);
        }
    }
    if (!early) {
        const int32_t* segs = a.unit_prefix + a.num_seqs + 1;
        carry = a.unit_prefix[a.num_seqs];
        seg_carry = segs[a.num_seqs];
        if (by_tile == 0) {
            const int64_t total = static_cast<int64_t>(carry) * a.H, line = total + static_cast<int64_t>(seg_carry) * extra;
            const int shares = dd_shares(total, grid);
            if (static_cast<int>(blockIdx.x) + 1 >= shares) return;
            // the unit of the boundary's tile
            const int cut = static_cast<int>(dd_tile_at(a.unit_prefix, segs, a.num_seqs, a.H, extra, dd_cut(line, extra, blockIdx.x + 1, shares), lo) / a.H);
            if (cut >= a.unit_prefix[lo + 1]) return;  // (the end of all)
            mt = (cut - a.unit_prefix[lo]) / dd_blocks(a.cache_lens[lo]);
        }
        begin = a.unit_prefix[lo];
        units = a.unit_prefix[lo + 1] - begin;
        seg_begin = segs[lo];
        s = dd_seq(a, lo);
    }
    if (units == 0 || mt >= s.tiles) return;
    if (!early) find_parts();
    // one share wrote it whole; the boundary lies between two of them, or an earlier one inside it has its CTA
    if (first == last || (by_tile == 0 && first != static_cast<int>(blockIdx.x))) return;
    const int count = last - first + 1;
    const int mine = warp % kShare, i_begin = count * mine / kShare, i_end = count * (mine + 1) / kShare;
    const int pairs = min(16, s.n * a.G - 16 * mt);
    constexpr int kAtOnce = kWarps / kShare;  // pairs
    for (int pair = blockIdx.z * kAtOnce + warp / kShare; pair < pairs; pair += gridDim.z * kAtOnce) {
        float m = -INFINITY, l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        // a part with no key (maximum -inf) weighs nothing, unless its sum is NaN
        auto weight = [](float2 ml, float top) {
            return ml.x == -INFINITY ? (ml.y == ml.y ? 0.f : ml.y) : dd_exp2(ml.x - top);
        };
        auto add = [&](float w, float2 ml, float4 v) {
            if (w != 0.f) {
                l = fmaf(w, ml.y, l);
                x.x = fmaf(w, v.x, x.x);
                x.y = fmaf(w, v.y, x.y);
                x.z = fmaf(w, v.z, x.z);
                x.w = fmaf(w, v.w, x.w);
            }
        };
        auto raise = [&](float top) {
            const float f = m == -INFINITY ? 0.f : dd_exp2(m - top);
            if (m != -INFINITY) {
                l *= f;
                x = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
            }
            m = top;
        };
        for (int i0 = i_begin; i0 < i_end; i0 += 8) {
            float4 v[8];
            float2 ml[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = min(i0 + u, i_end - 1);
                const int64_t at = (static_cast<int64_t>(i == 0 ? slot0 : 2 * (first + i)) * a.H + h) * 16 + pair;
                ml[u] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
                v[u] = *reinterpret_cast<const float4*>(a.part_o + at * kHeadDim + 4 * lane);
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < 8; ++u) top = fmaxf(top, ml[u].x);
            raise(top);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i0 + u < i_end) add(weight(ml[u], m), ml[u], v[u]);
        }
        if constexpr (kShare > 1) {
            static_assert(kShare == 1 || kAtOnce == 1, "the warps of a pair meet in block-wide barriers");
            sum_o[warp][lane] = x;
            if (lane == 0) sum_ml[warp] = make_float2(m, l);
            __syncthreads();
            if (warp == 0) {
                float top = m;
#pragma unroll
                for (int q = 1; q < kShare; ++q) top = fmaxf(top, sum_ml[q].x);
                raise(top);
#pragma unroll
                for (int q = 1; q < kShare; ++q) {
                    const float2 ml = sum_ml[q];
                    add(weight(ml, m), ml, sum_o[q][lane]);
                }
            }
        }
        if (mine == 0) {
            const float inv = 1.f / l;
            dd_store2(a, s, h, 16 * mt + pair, 4 * lane, x.x * inv, x.y * inv);
            dd_store2(a, s, h, 16 * mt + pair, 4 * lane + 2, x.z * inv, x.w * inv);
        }
        if constexpr (kShare > 1) __syncthreads();
    }
}

template <int H, bool kInt8, int kParts>
static cudaError_t launch_dense_decode(const DenseArgs& a, int grid, cudaStream_t stream) {
    using Cfg = DdCfg<kInt8>;
    const size_t smem = 1024 + static_cast<size_t>(Cfg::kStages) * Cfg::kStageBytes + Cfg::kMergeBytes +
                        2 * kDdPrefix * sizeof(int32_t);
    auto* kernel = dense_decode_kernel<H, kInt8, kParts>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kDdThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, *a.k_map, *a.v_map, a)) != cudaSuccess) return e;
    // tiles or boundaries, heads, (row, head) pairs
    const int tiles = (a.pairs_most + 15) / 16, pairs = std::min(16, a.pairs_most);
    const int by_tile = a.num_seqs * tiles <= grid ? tiles : 0;
    // Few parts each: a warp a pair, so that the CTAs fit at once (64 sequences of 8 heads x 4 pairs: 2,048 CTAs were two
    // waves); many: eight warps a pair (sixteen fit two CTAs an SM, again two waves); else four.
    const int segments = a.num_seqs * tiles, share = by_tile == 0 ? 4 : (grid >= 12 * segments ? 8 : (grid < 4 * segments ? 1 : 4));
    cfg.gridDim = dim3(static_cast<unsigned>(by_tile > 0 ? segments : grid), static_cast<unsigned>(a.H),
                       by_tile > 0 && share > 1 ? pairs : (pairs + 3) / 4);
    cfg.blockDim = dim3(share == 8 ? 256 : 128, 1, 1);
    cfg.dynamicSmemBytes = 0;
    auto* combine = share == 8 ? dense_combine_kernel<256, 8> : (share == 4 ? dense_combine_kernel<128, 4> : dense_combine_kernel<128, 1>);
    return cudaLaunchKernelEx(&cfg, combine, a, grid, by_tile);
}

// CTAs for so many units: one a SM at most, and at least two tiles each (fewer parts to join, the same latency).
int dense_decode_shares(int64_t units, int H) {
    const int64_t sms = std::min(device_sm_count(), kDenseMaxShares);
    const int64_t n = std::min(units, std::max<int64_t>(1, units * H / 2));
    return static_cast<int>(n < 1 ? 1 : (n < sms ? n : sms));
}

template <int H>
static cudaError_t launch_dense_decode_h(const DenseArgs& a, int grid, cudaStream_t stream) {
    if (a.kv_int8)
        return a.out_bf16 ? launch_dense_decode<H, true, 1>(a, grid, stream) : launch_dense_decode<H, true, 2>(a, grid, stream);
    return a.out_bf16 ? launch_dense_decode<H, false, 2>(a, grid, stream) : launch_dense_decode<H, false, 3>(a, grid, stream);
}

cudaError_t run_dense_decode(const DenseArgs& a, int shares, cudaStream_t stream) {
    switch (a.H) {
        case 1: return launch_dense_decode_h<1>(a, shares, stream);
        case 2: return launch_dense_decode_h<2>(a, shares, stream);
        case 4: return launch_dense_decode_h<4>(a, shares, stream);
        case 8: return launch_dense_decode_h<8>(a, shares, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace msa
