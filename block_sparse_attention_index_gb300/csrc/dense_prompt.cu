// Attention over every cached position on tcgen05: prompt chunks (more than 8 rows a sequence), causal, packed, with
// cached prefixes; and windows of several drafted rows.
//   out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m),  x_t = scale log2(e) q.k_t over t <= p
// in one pass over the keys with a running maximum.
//
// The G query heads of a KV head and P = 128 / G neighbouring positions make the 128 rows of an M tile (row = position
// x G + head), so a tile's rows share every key and value and the causal edge crosses few key tiles.  A CTA holds two
// such tiles ("stages") and walks the keys in tiles of NK:
//   S_s[128, NK] = Q_s K^T     both operands from shared memory (TMA, 128-byte swizzle), S in tensor memory
//   P_s = 2^(x - m)            softmax group s: one thread a row, S read from and P written over tensor memory
//   O_s[128, 128] += P_s V     P from tensor memory, V as it lies ([key][dim], MN-major), O in tensor memory
// While group 0 works on S_0 the tensor cores run P_1 V and S_1, and the other way round: 2,048 tensor cycles and two
// softmax passes of 128 x 128 a tile pair.  Tensor memory is full: S_0, S_1, O_0, O_1 of 128 columns each.  Each stage
// has an issuing thread of its own: the tensor pipe queues little, so a thread's test of a barrier (75 cycles even
// where the barrier is complete) or commit would leave it idle, eight of them in a pair's 32 instructions.  The two
// take turns, so that one stage's softmax falls into the other's products (left alone they fall into step: both
// softmaxes, then both stages' products).
//
// The running maximum is only raised when it would grow by more than 8 (a factor of 256 in the weights, which fp32
// sums and bf16 weights carry without loss); the group that owns O then multiplies it in tensor memory.  So most tiles
// rescale nothing.
//
// With bf16 outputs a weight enters P V as one bf16, 2^-8 of itself off at most and at random: in the 2-norm 1.66e-3 to
// 1.8e-3 of the outputs with their own rounding, which alone is 1.65e-3.  (A row with two keys may be off by 4.5e-3, more
// than fp32 outputs allow and less than a step of bf16, 7.8e-3 at 1.)  With
// fp32 outputs as three parts (2^-24), NK = 64 then, so that the parts fit over S.  The tensor cores cut what an
// addition loses instead of rounding it, a bias of about 2^-24 per addition of 16 keys (1.5e-4 after 33,280 keys,
// measured), so with fp32 outputs O_s holds two key tiles' products only and the softmax group adds them to its rows in
// registers; with bf16 outputs (whose half step is 2^-8) 256 tiles' products, which the group then adds to a sum in the
// workspace.
//
// Drafted windows (kAlt): one M tile, and the two stages take alternate key tiles, each with its own running state.
//
// One CTA per SM stays for the launch and takes items (a tile pair and a head), the longest first, as it gets through
// them (a counter; what an item holds and how it is computed does not depend on who has it).  Barriers, tensor memory and
// the ring of tiles run on from item to item: the next item's first copies and scores run under the last one's epilogue
// (a CTA for each item: 890 against 813 us for 4,096 rows at 8,192, 131 against 103 for eight packed prompts of 1 to
// 2,047 rows).  Items of the last wave, which would leave SMs idle, are split over their keys as well and their parts
// joined by dense_join_kernel.
//
// K and V are copied by two warps, 64 dimensions each: a thread's copies go out at about 48 B a cycle and a slot of the
// ring is free for one key tile's time, so with one thread the matrix instructions waited 580 of 2,900 cycles a tile for
// them (two: 300, which is what testing two complete barriers takes).
//
// What bounds it: bf16, the tensor pipe (4,096 rows at 8,192, 4 x 16 heads: 1.37 TFLOP in 800 to 880 us with the clocks
// that the power limit leaves, 1.56 to 1.71 PFLOP/s of 1.92 measured for cuBLAS in short bursts, 1.74 sustained); int8
// with bf16 outputs, the softmax groups' instructions (0.62 TFLOP in 518 us); fp32 outputs, likewise (0.55 TFLOP, with
// three weight parts 1.1 on the tensor cores, in 965 us); short sequences, the 3.5 us an item that its groups spend between
// its last scores and the next one's first, against 1.6 us a key tile.
//
// int8 caches are read from a copy widened once per call.  bf16 outputs: f16 values with the scales in them, over a
// power of two for each 64-position block (run_widen_f16), queries as f16 times a power of two for each row (converted
// in shared memory by the softmax threads; bf16's 8 bits fit, what lies 2^-22 below the row's largest loses some) and
// weights as one f16 (2^-11), at most 2^14: the blocks' powers of two are two scalars each for the softmax, where the
// scales themselves, one for each key, were a third of its instructions (784 us for 2,048 rows at 8,192, now 518).  fp32 outputs:
// bf16 integers, exact, scales beside them (run_widen_kv); the key scale multiplies the score, the value scale the weight.
// The rounded keys cost the outputs 1.75e-3 where their own rounding is 1.65e-3 (2-norm), with even keys as with one
// channel 16 times the others.  Rows whose blocks' scales lie too far apart for f16 are computed again, as below.
//
// Values that no row of the tile may see: positions past the length are zeroed in the last value tile (by warp 10), so
// stale cache rows do not matter.  A later token of the same chunk meets weights of zero; if its value is not finite
// the product is NaN, so a row whose result is not finite is computed again (dp_rows_again) where such a token lies past
// it in the item's tiles.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tensor_rows.cuh"

namespace msa {

constexpr int kDpThreads = 384;  // softmax groups: warps 0-3, 4-7; 8 and 10 copies, 9 and 11 matrix instructions
constexpr int kDpQBytes = 128 * kHeadDim * 2;
constexpr int kDpScaleSlots = 4;
constexpr float kDpSlack = 8.f;  // log2 by which the running maximum may lag

// A CTA's work: one of the launch's items (an M tile pair, kAlt: a single tile, of a sequence; and a KV head), whole or
// a part of its key range.
struct DpItem {
    int b, tile, h;            // b < 0: none
    int c0, n, L;              // of the sequence: first row, rows, length
    int split, nsplit, part;   // part `split` of `nsplit`; the part's place in the workspace
};
constexpr int kDpInfo = 3;     // items published ahead
constexpr int kDpClaim = 4;    // key tiles before the end of an item's copies at which the next one is taken

// Key tiles whose products O is summed over in tensor memory before they are added to the row's sum.
template <int kParts>
constexpr int kDpRun = kParts > 1 ? 2 : kDenseRunKeys / 128;

enum DpForm { kDpBf16 = 0, kDpInt = 1, kDpF16 = 2 };  // bf16 caches; int8: bf16 integers with scales; int8: f16 copy

template <int kParts, int kForm>
struct DpCfg {
    static constexpr int NK = kParts == 1 ? 128 : 64;
    static constexpr int kTile = NK * kHeadDim * 2;  // bytes of a K or V tile
    static constexpr int kStages = (kForm == kDpInt ? 4 : 5) * (128 / NK);
    // Column of S in its 128.  P's parts lie at columns 0, 32 and 64: with S from 64 on (fp32 outputs) a row's first 32
    // scores can be read, made into weights and overwritten before its last 32 are read.
    static constexpr int kSAt = kParts == 1 ? 0 : 64;
};

template <int kParts, int kForm>
struct __align__(1024) DpSmem {
    using Cfg = DpCfg<kParts, kForm>;
    static constexpr bool kWide = kForm == kDpInt;
    uint8_t q[2][kDpQBytes];
    uint8_t ring[Cfg::kStages][Cfg::kTile];
    float sc[kWide ? kDpScaleSlots : 1][2][kWide ? 128 : 4];  // key and value scales of a tile
    // Copies landed.  Two stages a tile: [0][ring slot], every slot seen by both issuers.  Alternate tiles: issuer s's
    // n-th copy completes [s][n % kStages], so that each issuer sees its barriers' phases one after the other (a slot's
    // phases would belong to either, and a wait that skipped one could not tell by parity that it had).
    uint64_t full[2][Cfg::kStages], empty[Cfg::kStages];
    uint64_t sc_full[kDpScaleSlots], sc_empty[kDpScaleSlots];
    uint64_t v_last[Cfg::kStages];       // a last value tile has landed, before its tail is zeroed
    uint64_t q_full, q_turned[2], q_empty;  // q_turned: a stage's queries converted (f16 form)
    uint64_t s_full[2], p_full[2][2], o_full[2], turn[2], drain[2];  // P: by halves of the key tile
    uint32_t tmem, lost;  // lost: some block of the f16 copy has lost bits
    int32_t scan[kDpThreads / 32];
    float scan_keys[kDpThreads / 32];
    DpItem info[kDpInfo];  // the CTA's next items, published by warp 10
    uint64_t info_full[kDpInfo], info_empty[kDpInfo];
    uint64_t item_done;  // both issuers are through with an item
    float2 other_ml[128];  // drafted windows: maxima and sums of the second stream
};
static_assert(sizeof(DpSmem<1, kDpBf16>) + 1024 <= 227 * 1024, "prompt attention exceeds 227 KB of shared memory");
static_assert(sizeof(DpSmem<1, kDpF16>) + 1024 <= 227 * 1024, "prompt attention (f16 copy) exceeds 227 KB of shared memory");
static_assert(sizeof(DpSmem<3, kDpInt>) + 1024 <= 227 * 1024, "prompt attention (int8, fp32) exceeds 227 KB of shared memory");
static_assert(sizeof(DpSmem<3, kDpBf16>) + 1024 <= 227 * 1024, "prompt attention (fp32) exceeds 227 KB of shared memory");

// A barrier of the 256 softmax threads that returns the AND of p.
__device__ __forceinline__ bool dp_sync_and(bool p) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q, o;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.and.pred o, 1, 256, q;\n\t"
                 "selp.u32 %0, 1, 0, o;\n\t}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(p))
                 : "memory");
    return r != 0;
}
// Items of the sequence without its heads; its metadata; `keys`: its items' key tiles (128 positions).
template <bool kAlt>
__device__ __forceinline__ int dp_tiles(const DenseArgs& a, int b, DpItem& it, float& keys, bool& bad) {
    bad = false;
    keys = 0.f;
    // (loads that need not wait for one another)
    const int c0 = a.cu_rows[b], n = a.cu_rows[b + 1] - c0, L = a.cache_lens[b];
    const bool placed = seq_rows_ok(a.seq_cache, b, L, a.seq_cache_tokens);
    const bool here = a.cache.table != nullptr || a.cache.starts[b] >= 0;  // (else widened in another pass)
    if (n == 0) return 0;
    if (kAlt ? n < 0 || n > kDecodeMaxRows || n * a.G <= a.window_above : a.only_multi_row && n > 0 && n <= kDecodeMaxRows) return 0;
    if (n < 0 || n > a.max_rows_per_seq || c0 < 0 || c0 + n > a.total_rows || L < n || L > a.max_cache_len || !placed) {
        bad = true;
        return 0;
    }
    if (!here) return 0;
    it.c0 = c0;
    it.n = n;
    it.L = L;
    const int rows = (128 / a.G) * (kAlt ? 1 : 2), tiles = (n + rows - 1) / rows;
    keys = tiles * (static_cast<float>(L) - 0.5f * n) * (1.f / 128.f);
    return tiles;
}

// What `n` parts of each of the last wave's `rest` items cost, in key tiles: a wave of CTAs takes its tiles and what a
// CTA costs besides (about six; parts ten, as they write 32-bit rows), and the parts are joined.
__host__ __device__ constexpr float dp_cost(int rest, int places, float tiles, int n) {
    return ((rest * n + places - 1) / places) * (tiles / n + (n > 1 ? 10.f : 6.f)) + (n > 1 ? 12.f : 0.f);
}

// Key ranges that the items of the last, unfilled wave are split into: `rest` items of `tiles` key tiles each on `places`
// SMs, `most` parts at most; lane n - 1 weighs n parts.
__device__ __forceinline__ int dp_split(int rest, int places, float tiles, int most) {
    const int n = (threadIdx.x & 31) + 1;
    const bool fits = n == 1 || (rest > 0 && rest * n <= most && tiles >= 4.f * n);
    const uint32_t mine = fits ? static_cast<uint32_t>(dp_cost(rest, places, tiles, n) * 16.f) << 5 | (n - 1) : 0xffffffffu;
    return static_cast<int>(__reduce_min_sync(0xffffffffu, mine) & 31u) + 1;
}

// The launch's items: all sequences' tiles counted by the block.  Whole waves of items go whole; those of the last wave
// may be split.
struct DpPlan {
    int total, all, whole, nsplit;  // tiles; items; items that go whole; parts of the others
    int before, mine;               // up to 32 sequences: of sequence `lane`, the tiles before it and its own
    DpItem seq;                     // and its metadata
};
template <bool kAlt, int kThreads>
__device__ DpPlan dp_plan(const DenseArgs& a, int items, int32_t* scan, float* scan_keys) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool few = a.num_seqs <= 32;  // every warp counts by itself, a lane a sequence
    const int per = (a.num_seqs + kThreads - 1) / kThreads, at = few ? lane : tid;
    const int b0 = min(at * per, a.num_seqs), b1 = min(b0 + per, a.num_seqs);
    DpPlan p{};
    float keys = 0.f;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        float k;
        p.mine += dp_tiles<kAlt>(a, b, p.seq, k, bad);
        keys += k;
        if (bad && blockIdx.x == 0) atomicOr(a.err, kErrBadMetadata);
    }
    int incl = p.mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) keys += __shfl_xor_sync(0xffffffffu, keys, o);
    p.before = incl - p.mine;
    p.total = __shfl_sync(0xffffffffu, incl, 31);
    if (!few) {
        if (lane == 31) scan[warp] = incl;
        if (lane == 0) scan_keys[warp] = keys;
        __syncthreads();
        p.total = 0;
        keys = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) p.before += scan[w];
            p.total += scan[w];
            keys += scan_keys[w];
        }
        // the tiles before each sequence, for the search (every CTA writes the same)
        int before = p.before;
        for (int b = b0; b < b1; ++b) {
            bool bad;
            float k;
            DpItem it;
            a.tile_prefix[b] = before;
            before += dp_tiles<kAlt>(a, b, it, k, bad);
        }
    }
    // more tiles than the host's row counts allow for: the first of them go without
    if (p.total > items && blockIdx.x == 0 && tid == 0) atomicOr(a.err, kErrBadMetadata);
    p.all = min(p.total, items) * a.H;
    p.whole = p.all / a.places * a.places;
    const int rest = p.all - p.whole;
    p.nsplit = dp_split(rest, a.places, p.total > 0 ? keys / p.total : 0.f, a.parts_most);
    if (blockIdx.x == 0 && tid == 0) *a.split_head = make_int2(p.nsplit > 1 ? rest : 0, p.nsplit);
    return p;
}

// Work g of the launch (a whole warp): its item, the longest first (the last tile of a sequence has the most keys).
__device__ DpItem dp_find(const DenseArgs& a, const DpPlan& p, int g) {
    const int lane = threadIdx.x & 31, r = g - p.whole;
    DpItem x{};
    x.b = -1;
    const int item = r < 0 ? g : p.whole + r / p.nsplit;
    if (item >= p.all) return x;
    const int want = p.total - 1 - item / a.H;
    if (a.num_seqs <= 32) {
        const uint32_t who = __ballot_sync(0xffffffffu, want >= p.before && want < p.before + p.mine);
        const int from = __ffs(who) - 1;
        x.b = from;
        x.tile = want - __shfl_sync(0xffffffffu, p.before, from);
        x.c0 = __shfl_sync(0xffffffffu, p.seq.c0, from);
        x.n = __shfl_sync(0xffffffffu, p.seq.n, from);
        x.L = __shfl_sync(0xffffffffu, p.seq.L, from);
    } else {
        int lo = 0, hi = a.num_seqs;  // largest b with tile_prefix[b] <= want, 32 candidates at a time
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const uint32_t le = __ballot_sync(0xffffffffu, at < hi && a.tile_prefix[at] <= want);
            lo += (31 - __clz(le)) * step;
            hi = min(lo + step, hi);
        }
        x.b = lo;
        x.tile = want - a.tile_prefix[lo];
        x.c0 = a.cu_rows[lo];
        x.n = a.cu_rows[lo + 1] - x.c0;
        x.L = a.cache_lens[lo];
    }
    x.h = item % a.H;
    x.nsplit = r < 0 ? 1 : p.nsplit;
    x.split = r < 0 ? 0 : r % p.nsplit;
    x.part = r;
    if (x.nsplit > 1 && x.split == 0 && lane == 0) a.split_items[item - p.whole] = make_int4(x.b, x.tile, x.h, 0);
    return x;
}

// What an item covers.
struct DpWork {
    int b, c0, n, L, i0;      // sequence, its first row, rows, length; first row of the item in the sequence
    int P;                    // positions of an M tile
    int first;                // first key tile of this part
    int count[2];             // key tiles of each stage
    int total;                // key tiles loaded
};

template <bool kAlt, int NK>
__device__ __forceinline__ DpWork dp_work(int P, const DpItem& it) {  // P = 128 / G
    DpWork w;
    w.b = it.b;
    w.c0 = it.c0;
    w.n = it.n;
    w.L = it.L;
    w.P = P;
    w.i0 = it.tile * w.P * (kAlt ? 1 : 2);
    const int p0 = w.L - w.n;
    // keys up to the last row of each M tile
    const int end0 = p0 + min(w.n, w.i0 + w.P), end1 = p0 + min(w.n, w.i0 + 2 * w.P);
    const int all = (max(end0, end1) + NK - 1) / NK;
    int last = all;
    w.first = 0;
    if (it.nsplit > 1) {  // (at most 2^15 tiles and 32 parts)
        w.first = static_cast<int>(static_cast<uint32_t>(all) * it.split / it.nsplit);
        last = static_cast<int>(static_cast<uint32_t>(all) * (it.split + 1) / it.nsplit);
    }
    w.total = last - w.first;
    if (kAlt) {
        w.count[0] = (w.total + 1) / 2;
        w.count[1] = w.total / 2;
    } else {
        w.count[0] = max(0, min(last, (end0 + NK - 1) / NK) - w.first);
        w.count[1] = w.i0 + w.P < w.n ? w.total : 0;
        w.total = max(w.count[0], w.count[1]);
    }
    return w;
}

// Up to four rows of a warp again over keys [first, end[r]), in fp32: where a product with a later token's infinite or NaN
// value spoiled them, or the f16 copy's powers of two left them too few bits.  The whole warp, 32 keys at a time: 16
// lanes share a key's dot products (8 dimensions each, summed by a reduce-scatter over 16 keys), then a lane has a key's
// scores; 4 dimensions of O a lane.  70 cycles a key and row, bound by the instructions (one row at a time, loads in the
// order of its keys: 710).  A warp's 32 rows over 2^21 keys take 2.5 s, so the CTA's other warps
// may wait longer for them than kWaitLimitNs: kDpAgainNs more for each key.
constexpr int kDpAgain = 4;
constexpr uint64_t kDpAgainNs = 8000;  // 32 rows x 70 cycles are 1.2 us; two warps a scheduler, low clocks, one stage after the other
struct DpAgain {
    int64_t q_row[kDpAgain];
    int end[kDpAgain];
    float o[kDpAgain][4], m[kDpAgain], l[kDpAgain];
};
template <bool kInt8>
__device__ __noinline__ void dp_rows_again(const DenseArgs& a, int b, int h, int first, DpAgain& g) {
    const int lane = threadIdx.x & 31, dl = lane & 15;
    float q[kDpAgain][8], o[kDpAgain][4], m[kDpAgain], l[kDpAgain];
    int end[kDpAgain], last = 0;
#pragma unroll
    for (int r = 0; r < kDpAgain; ++r) {
        const uint4 w = *reinterpret_cast<const uint4*>(a.q + g.q_row[r] * kHeadDim + 8 * dl);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q[r][2 * e] = bf16_lo(ws[e]);
            q[r][2 * e + 1] = bf16_hi(ws[e]);
            o[r][e] = 0.f;
        }
        m[r] = -INFINITY;
        l[r] = 0.f;
        end[r] = g.end[r];
        last = max(last, end[r]);
    }
    for (int u0 = first; u0 < last; u0 += 32) {
        const int t = u0 + lane;
        int64_t row = 0;  // (past the last key: row 0, not added)
        float kf = a.scale_log2, vf = 1.f;
        if (t < last) {
            const int64_t base = block_row(a.seq_cache, b, t & ~(kBlock - 1));
            row = base < 0 ? 0 : (base + (t & (kBlock - 1))) * a.H + h;
            if constexpr (kInt8) {
                kf *= a.seq_k_scale[row];
                vf = a.seq_v_scale[row];
            }
        }
        float acc[kDpAgain][16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {  // keys i and 16 + i
            const int64_t at = __shfl_sync(0xffffffffu, row, i + (lane & 16)) * kHeadDim + 8 * dl;
            float k[8];
            if constexpr (kInt8) {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(a.k) + at);
#pragma unroll
                for (int e = 0; e < 8; ++e) k[e] = static_cast<float>(static_cast<int8_t>((e < 4 ? w.x : w.y) >> (8 * (e & 3))));
            } else {
                const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k) + at);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) k[e] = e & 1 ? bf16_hi(ws[e >> 1]) : bf16_lo(ws[e >> 1]);
            }
#pragma unroll
            for (int r = 0; r < kDpAgain; ++r) {
                float x = k[0] * q[r][0];
#pragma unroll
                for (int e = 1; e < 8; ++e) x = fmaf(k[e], q[r][e], x);
                acc[r][i] = x;
            }
        }
        float p[kDpAgain];
#pragma unroll
        for (int r = 0; r < kDpAgain; ++r) {
#pragma unroll
            for (int d = 8; d > 0; d >>= 1)
#pragma unroll
                for (int i = 0; i < d; ++i) {
                    const float send = dl & d ? acc[r][i] : acc[r][i + d], keep = dl & d ? acc[r][i + d] : acc[r][i];
                    acc[r][i] = keep + __shfl_xor_sync(0xffffffffu, send, d);
                }
            const float x = t < end[r] ? acc[r][0] * kf : -INFINITY;
            float top = x;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(top, m[r]);
            const float f = m[r] == -INFINITY ? 0.f : dp_exp2(m[r] - top);
            p[r] = t < end[r] ? dp_exp2(x - (top == -INFINITY ? 0.f : top)) : 0.f;  // (no score above -inf so far: weights of 0)
            l[r] *= f;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][e] *= f;
            m[r] = top;
        }
        for (int i0 = 0; i0 < 32 && u0 + i0 < last; i0 += 16) {  // sixteen values in flight
            float v[16][4];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t at = __shfl_sync(0xffffffffu, row, i0 + i) * kHeadDim + 4 * lane;
                if constexpr (kInt8) {
                    const char4 w = *reinterpret_cast<const char4*>(static_cast<const int8_t*>(a.v) + at);
                    const float f = __shfl_sync(0xffffffffu, vf, i0 + i);
                    v[i][0] = w.x * f;
                    v[i][1] = w.y * f;
                    v[i][2] = w.z * f;
                    v[i][3] = w.w * f;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.v) + at);
                    v[i][0] = bf16_lo(w.x);
                    v[i][1] = bf16_hi(w.x);
                    v[i][2] = bf16_lo(w.y);
                    v[i][3] = bf16_hi(w.y);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int r = 0; r < kDpAgain; ++r) {
                    const float w = __shfl_sync(0xffffffffu, p[r], i0 + i);
                    if (u0 + i0 + i < end[r]) {
                        l[r] += w;
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[r][e] = fmaf(w, v[i][e], o[r][e]);
                    }
                }
        }
    }
#pragma unroll
    for (int r = 0; r < kDpAgain; ++r) {
        g.m[r] = m[r];
        g.l[r] = l[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) g.o[r][e] = o[r][e];
    }
}

// The last of the positions [first, end) whose value is not finite, -1 if all are (a whole warp).
__device__ __noinline__ int dp_last_bad(const DenseArgs& a, int b, int h, int first, int end) {
    int bad = -1;
    for (int t = first + static_cast<int>(threadIdx.x & 31); t < end; t += 32) {
        int64_t row = block_row(a.seq_cache, b, t & ~(kBlock - 1));
        if (row < 0) continue;
        row = (row + (t & (kBlock - 1))) * a.H + h;
        bool is = false;
        if (a.kv_int8) {
            is = !(fabsf(a.seq_v_scale[row]) < INFINITY);
        } else {
            const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v) + row * kHeadDim);
#pragma unroll 4
            for (int i = 0; i < kHeadDim / 8; ++i) {
                const uint4 x = v[i];
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) is |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
            }
        }
        if (is) bad = t;
    }
    return __reduce_max_sync(0xffffffffu, bad);
}

// bf16 outputs: the row's sum over earlier runs of tiles lies in the workspace, [128 dims, maximum, value exponent][row] of
// the CTA's stage.  Adds O in tensor memory to it (`first`: there was none) or, `back`, it to O (a whole warp, a row a
// thread), in units of the present maximum and value exponent.
constexpr int kDpAsideRows = kHeadDim + 2;
__device__ __forceinline__ void dp_aside(float* base, uint32_t o_addr, float top, int vexp, bool first, bool back) {
    float* aside = base + (static_cast<int64_t>(blockIdx.x) * 2 + (threadIdx.x >> 7)) * (kDpAsideRows * 128) + (threadIdx.x & 127);
    float f = 0.f;
    if (!first) {
        const float then = aside[kHeadDim * 128];
        const int e = static_cast<int>(aside[(kHeadDim + 1) * 128]) - vexp;
        f = then == -INFINITY || e < -126 ? 0.f : dp_exp2(then - top) * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    }
#pragma unroll 1
    for (int q = 0; q < kHeadDim / 32; ++q) {
        float y[32];
        dp_ld32(o_addr + 32 * q, y);
        tmem_ld_wait();
        if (!first) {
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = fmaf(aside[(32 * q + k) * 128], f, y[k]);
        }
        if (back) {
            dp_st32(o_addr + 32 * q, reinterpret_cast<const uint32_t*>(y));
        } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) aside[(32 * q + k) * 128] = y[k];
        }
    }
    if (back) {
        dp_st_wait();
    } else {
        aside[kHeadDim * 128] = top;
        aside[(kHeadDim + 1) * 128] = static_cast<float>(vexp);
    }
}

// The same as a call, which is what the kernel on bf16 caches runs faster with (8 packed prompts 106 us, inline 108), and
// the one on the f16 copy slower (2,048 rows at 8,192 531, inline 518).
__device__ __noinline__ void dp_aside_call(float* base, uint32_t o_addr, float top, int vexp, bool first, bool back) {
    dp_aside(base, o_addr, top, vexp, first, back);
}

// How far apart the value factors of an item's blocks are, log2 (blocks of zeros left out); 127 if some key or value of
// one has lost bits (a whole warp).
__device__ __noinline__ int dp_apart(const float2* fac, int first, int end) {
    int most = 0, least = 255, lost = 0;
    for (int b = first + static_cast<int>(threadIdx.x & 31); b < end; b += 32) {
        const float2 f = fac[b];
        const int e = static_cast<int>(__float_as_uint(f.y) >> 23);
        lost |= static_cast<int>(__float_as_uint(f.x) & 1u);
        most = max(most, e);
        if (e > 0) least = min(least, e);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    return __any_sync(0xffffffffu, lost) ? 127 : most - least;
}

template <int kParts, int kForm, bool kAlt>
__global__ void __launch_bounds__(kDpThreads, 1) dense_prompt_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                    const __grid_constant__ CUtensorMap k_map,
                                                                    const __grid_constant__ CUtensorMap v_map,
                                                                    const DenseArgs a, int items) {
    constexpr bool kWide = kForm == kDpInt, kF16 = kForm == kDpF16;
    using Cfg = DpCfg<kParts, kForm>;
    constexpr int NK = Cfg::NK, kStages = Cfg::kStages, kHalf = Cfg::kTile / 2, kSAt = Cfg::kSAt;
    extern __shared__ uint8_t smem_raw[];
    using Smem = DpSmem<kParts, kForm>;
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, a.err, a.wait_ns); };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be scheduled: it waits for this grid
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[0][s], 2);  // two warps copy a half each
            mbar_init(&sm.full[1][s], 2);
            mbar_init(&sm.v_last[s], 2);
            mbar_init(&sm.empty[s], kAlt ? 1 : 2);  // the stages' issuers (one with fewer tiles lets the others pass)
        }
        for (int s = 0; s < kDpScaleSlots; ++s) {
            mbar_init(&sm.sc_full[s], 1);
            mbar_init(&sm.sc_empty[s], 8);
        }
        for (int s = 0; s < kDpInfo; ++s) {
            mbar_init(&sm.info_full[s], 1);
            mbar_init(&sm.info_empty[s], 11);  // copies, two issuers, eight softmax warps
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, kAlt ? 6 : 2);  // two issuers; kAlt: and group 0, whose epilogue uses the query buffers
        mbar_init(&sm.item_done, 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.q_turned[s], 4);
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.p_full[s][0], 4);
            mbar_init(&sm.p_full[s][1], 4);
            mbar_init(&sm.o_full[s], 1);
            mbar_init(&sm.turn[s], 1);
            mbar_init(&sm.drain[s], 1);
        }
        fence_mbar_init();
    }
    if (kF16 && tid == 0) sm.lost = *a.wide_lost;
    if (warp == 8 && lane < 3) prefetch_tmap(lane == 0 ? &q_map : (lane == 1 ? &k_map : &v_map));
    if (warp == 9) tmem_alloc(&sm.tmem, 512);
    tc_fence_before();
    const DpPlan plan = dp_plan<kAlt, kDpThreads>(a, items, sm.scan, sm.scan_keys);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int P = 128 / a.G;

    // Every role walks the CTA's items with its own copy of each and with counts that run on over them: copies (ring slots),
    // a stage's copies (alternate tiles), a stage's tiles, items.
    auto next_item = [&](int k, DpItem& x) {  // item k of the CTA, false where it never came
        if (!wait(&sm.info_full[k % kDpInfo], (k / kDpInfo) & 1)) return false;
        x = sm.info[k % kDpInfo];
        return true;
    };
    // the value tile that holds the end of the sequence, if its last rows are nobody's
    auto last_tile = [&](const DpWork& w) {
        const int v_end = w.L / NK;
        return w.L % NK != 0 && v_end >= w.first && v_end < w.first + w.total ? v_end - w.first : -1;
    };
    // tile j's K (0) or V (1) among the copies of an item (alternate tiles: of its stage)
    auto copy_index = [&](int j, int kind) { return kAlt ? 2 * (j >> 1) + kind : 2 * j + kind; };
    auto full_bar = [&](int j, int n) { return &sm.full[kAlt ? j & 1 : 0][n % kStages]; };  // n: running copy index
    // ring slots of an item's key tile j: K0 V0 K1 V1 ..., or (alternate tiles) K0 K1 V0 K2 V1 ...
    auto slot_k = [&](int j) { return kAlt ? (j == 0 ? 0 : 2 * j - 1) : 2 * j; };
    auto slot_v = [&](const DpWork& w, int j) { return kAlt ? (j + 1 < w.total ? 2 * j + 2 : 2 * j + 1) : 2 * j + 1; };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8 || warp == 10) {
            // ---------------- copies: K and V tiles in the order the matrix instructions take them, dimensions 0-63 by warp 8
            // (and the queries and scales), 64-127 by warp 10 (and items and last value tiles)
            const int half = warp == 10;
            int slot = 0, sent[2] = {0, 0}, tiles_before = 0, queries = 0;  // copies so far, by barrier row; key tiles; items
            uint32_t fixed = 0;  // last value tiles, a bit a ring slot: how often modulo 2
            bool alive = true;
            DpItem item, after;
            auto publish = [&](int n, const DpItem& x) {  // item n of the CTA
                int ok = 1;
                if (lane == 0) {
                    const int at = n % kDpInfo;
                    if (n >= kDpInfo) ok = wait(&sm.info_empty[at], ((n / kDpInfo) - 1) & 1);
                    if (ok) {
                        sm.info[at] = x;
                        mbar_arrive(&sm.info_full[at]);
                    }
                }
                return __shfl_sync(0xffffffffu, ok, 0) != 0;
            };
            if (half) {
                after = dp_find(a, plan, blockIdx.x);
                alive = publish(0, after);
            }
            for (int k = 0; alive; ++k) {
                if (half) {
                    item = after;
                } else {
                    alive = __all_sync(0xffffffffu, next_item(k, item));
                    if (!alive) break;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.info_empty[k % kDpInfo]);
                }
                if (item.b < 0) break;
                const DpWork w = dp_work<kAlt, NK>(P, item);
                const int h = item.h, fix = last_tile(w);
                if (!half) {
                    int ok = 1;
                    if (lane == 0) {
                        if (k > 0) ok = wait(&sm.q_full, (k - 1) & 1) && wait(&sm.q_empty, (k - 1) & 1);
                        if (ok) {
                            const int tiles = kAlt ? 1 : (w.i0 + w.P < w.n ? 2 : 1);
                            mbar_arrive_expect_tx(&sm.q_full, tiles * 2 * w.P * a.G * 128);
                            for (int s = 0; s < tiles; ++s)
                                for (int c = 0; c < 2; ++c)
                                    tma_load_3d(sm.q[s] + c * (kDpQBytes / 2), &q_map, &sm.q_full, 64 * c, h * a.G, w.c0 + w.i0 + s * w.P);
                            ++queries;
                        }
                    }
                    alive = __shfl_sync(0xffffffffu, ok, 0) != 0;
                }
                const int sent0[2] = {sent[0], sent[1]};
                int64_t row = 0;
                // a copy step i loads K tile i (if any) and V tile i - lag: the order K0 V0 K1 V1 ... (two stages a tile) or
                // K0 K1 V0 K2 V1 ... (alternate tiles)
                constexpr int kLag = kAlt ? 1 : 0;
                constexpr int kBatch = 32 / (NK / kBlock);  // tiles whose cache rows the lanes hold
                int64_t row_before = 0;                     // the previous batch's (a V tile may still need its last one)
                const int claim_at = max(0, w.total - kDpClaim);
                for (int i = 0; alive && (i < w.total + kLag || i == 0); ++i) {
                    if (half && i == claim_at) {  // which CTA has which item is left to their timing, what an item holds is not
                        int g = 0;
                        if (lane == 0) g = gridDim.x + atomicAdd(a.next_item, 1u);
                        after = dp_find(a, plan, __shfl_sync(0xffffffffu, g, 0));
                        alive = publish(k + 1, after);
                        if (!alive) break;
                    }
                    if (w.total == 0) break;
                    if (i % kBatch == 0) {
                        row_before = row;
                        const int64_t t = (static_cast<int64_t>(w.first) + i) * NK + lane * kBlock;
                        row = a.cache_tokens;  // past the length: a box past the cache is zeros
                        if (t < w.L && t < static_cast<int64_t>(w.first + w.total) * NK) {
                            row = block_row(a.cache, w.b, t);
                            if (row < 0) {  // page outside the pool
                                atomicOr(a.err, kErrBadMetadata);
                                row = a.cache_tokens;
                            }
                        }
                    }
#pragma unroll
                    for (int kind = 0; kind < 2; ++kind) {  // K, V
                        const int j = kind == 0 ? i : i - kLag;
                        if (j < 0 || j >= w.total) continue;
                        const int st = slot % kStages;
                        const bool old = kind == 1 && kLag == 1 && i % kBatch == 0;
                        int64_t r[NK / kBlock];
#pragma unroll
                        for (int c = 0; c < NK / kBlock; ++c)
                            r[c] = __shfl_sync(0xffffffffu, old ? row_before : row, (j % kBatch) * (NK / kBlock) + c);
                        int ok = 1;
                        if (lane == 0) {
                            // the last value tile completes a barrier of its own: warp 10 zeroes its tail and passes it on
                            const int odd = kAlt ? j & 1 : 0;
                            uint64_t* bar = kind == 1 && j == fix ? &sm.v_last[st]
                                                                  : full_bar(j, (odd ? sent0[1] : sent0[0]) + copy_index(j, kind));
                            uint8_t* dst = sm.ring[st] + half * kHalf;
                            if (slot >= kStages) ok = wait(&sm.empty[st], ((slot / kStages) - 1) & 1);
                            if (ok) {
                                mbar_arrive_expect_tx(bar, Cfg::kTile / 2);
#pragma unroll
                                for (int c = 0; c < NK / kBlock; ++c)
                                    tma_load_3d(dst + c * (kBlock * 128), kind == 0 ? &k_map : &v_map, bar, 64 * half, h, static_cast<int>(r[c]));
                                if (kWide && kind == 0 && !half) {  // the tile's scales
                                    const int jt = tiles_before + j, e = jt % kDpScaleSlots;
                                    if (jt >= kDpScaleSlots) ok = wait(&sm.sc_empty[e], ((jt / kDpScaleSlots) - 1) & 1);
                                    if (ok) {
                                        const int64_t from = static_cast<int64_t>(h) * a.cache_tokens + a.cache.starts[w.b] +
                                                             static_cast<int64_t>(w.first + j) * NK;
                                        mbar_arrive_expect_tx(&sm.sc_full[e], 2 * NK * 4);
                                        dp_bulk(sm.sc[e][0], a.k_scale + from, NK * 4, &sm.sc_full[e]);
                                        dp_bulk(sm.sc[e][1], a.v_scale + from, NK * 4, &sm.sc_full[e]);
                                    }
                                }
                            }
                        }
                        ++slot;
                        if (kAlt && (j & 1)) ++sent[1];
                        else ++sent[0];
                        if (!__shfl_sync(0xffffffffu, ok, 0)) {
                            alive = false;
                            break;
                        }
                    }
                }
                if (half && fix >= 0 && alive) {  // ---- the last value tile: rows past the length become zero
                    const int st = (2 * tiles_before + slot_v(w, fix)) % kStages;
                    alive = __all_sync(0xffffffffu, wait(&sm.v_last[st], fixed >> st & 1));
                    if (!alive) break;
                    fixed ^= 1u << st;
                    for (int x = (w.L % NK) * 16 + lane; x < NK * 16; x += 32) {
                        const int key = x >> 4, c = x & 15;  // 16-byte chunk c & 7 of half c >> 3 (a whole row: no swizzle to undo)
                        *reinterpret_cast<uint4*>(sm.ring[st] + (c >> 3) * kHalf + key * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        uint64_t* bar = full_bar(fix, sent0[kAlt ? fix & 1 : 0] + copy_index(fix, 1));
                        mbar_arrive(bar);
                        mbar_arrive(bar);
                    }
                }
                tiles_before += w.total;
            }
            if (lane == 0 && !half) {  // no copy in flight at the end (a last value tile's barrier was warp 10's to wait for)
                if (queries > 0) wait(&sm.q_full, (queries - 1) & 1);
                for (int s = 0; s < (kAlt ? 2 : 1); ++s)
                    for (int b = 0; b < kStages && b < sent[s]; ++b)
                        wait(&sm.full[s][b], ((sent[s] - 1 - b) / kStages) & 1);
                if (kWide && alive)
                    for (int e = 0; e < kDpScaleSlots && e < tiles_before; ++e)
                        wait(&sm.sc_full[e], ((tiles_before - 1 - e) / kDpScaleSlots) & 1);
            }
        } else if (warp == 9 || warp == 11) {
            // ---------------- matrix instructions of stage s, one thread
            const int s = warp == 9 ? 0 : 1;
            if (lane == 0) {
                constexpr uint32_t idesc_s = kF16 ? idesc_f16_f32(128, NK, 0) : idesc_bf16_f32(128, NK, 0, 0);
                constexpr uint32_t idesc_o = kF16 ? idesc_f16_f32(128, kHeadDim, 1) : idesc_bf16_f32(128, kHeadDim, 0, 1);
                const uint64_t qd = smem_desc_sw128(smem_u32(sm.q[kAlt ? 0 : s]), 16, 1024);
                const uint64_t kd = smem_desc_sw128(smem_u32(sm.ring[0]), 16, 1024);
                const uint64_t vd = smem_desc_sw128(smem_u32(sm.ring[0]), kHalf, 1024);
                constexpr int kStep = kAlt ? 2 : 1;
                const int j0 = kAlt ? s : 0;
                // running: ring slots, tiles of the stage, turns taken, the next copy's barrier and its phase
                int slots = 0, tiles = 0, turns = 0, bar = 0;
                uint32_t bar_phase = 0;
                auto landed = [&]() { return wait(&sm.full[kAlt ? s : 0][bar], bar_phase); };
                auto pass_copy = [&]() {
                    if (++bar == kStages) {
                        bar = 0;
                        bar_phase ^= 1;
                    }
                };
                bool ok = true, issued = false;
                for (int k = 0; ok; ++k) {
                    DpItem item;
                    ok = next_item(k, item);
                    if (!ok) break;
                    mbar_arrive(&sm.info_empty[k % kDpInfo]);
                    if (item.b < 0) break;
                    const DpWork w = dp_work<kAlt, NK>(P, item);
                    const int count = s == 0 ? w.count[0] : w.count[1], others = s == 0 ? w.count[1] : w.count[0];
                    // S_s = Q_s K^T from ring slot st; `pass`: the other stage's turn begins while the last of them run
                    auto scores = [&](int st, bool last, bool pass) {
                        const uint64_t kb = kd + static_cast<uint64_t>(st * (Cfg::kTile >> 4));
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            tc_mma_ss(tmem + s * 128 + kSAt, qd + static_cast<uint64_t>(((i >> 2) * (kDpQBytes / 2) + (i & 3) * 32) >> 4),
                                      kb + static_cast<uint64_t>(((i >> 2) * kHalf + (i & 3) * 32) >> 4), idesc_s, i > 0);
                            if (i == 5 && pass) mbar_arrive(&sm.turn[s ^ 1]);
                        }
                        tc_commit(&sm.s_full[s]);
                        if (!kAlt && last) tc_commit(&sm.q_empty);  // the last products with this item's queries
                        tc_commit(&sm.empty[st]);
                    };
                    // (waited for without tiles too: a barrier's phases have to be seen one by one, and the stage's group may
                    // be converting the queries)
                    ok = wait(kF16 ? &sm.q_turned[s] : &sm.q_full, k & 1);
                    if (!ok) break;
                    if constexpr (kAlt) mbar_arrive(&sm.q_empty);  // (seen; group 0 arrives when the products are done)
                    if (count > 0) {
                        ok = landed();
                        if (!ok) break;
                        issued = true;
                        tc_fence_after();
                        scores(kAlt ? (slots + slot_k(j0)) % kStages : bar, count == 1, false);
                        pass_copy();
                    } else if (!kAlt) {
                        mbar_arrive(&sm.q_empty);
                    }
                    // the other stage is through with its last item: its turns have been taken
                    if (k > 0) ok = wait(&sm.item_done, (k - 1) & 1);
                    for (int c = 0; ok && c < count; ++c) {
                        // the stages take turns: values of tile c, scores of the next (whatever can be waited for is, first)
                        const int j = j0 + kStep * c;
                        const uint32_t phase = (tiles + c) & 1;
                        const bool next = c + 1 < count;
                        ok = landed();
                        const int st_v = kAlt ? (slots + slot_v(w, j)) % kStages : bar;
                        pass_copy();
                        ok = ok && (!next || landed());
                        const int st_k = kAlt ? (slots + slot_k(j + kStep)) % kStages : bar;
                        if (next) pass_copy();
                        const bool turns_now = s == 0 ? c > 0 && c <= others : c < others;
                        const bool pass = s == 0 ? c < others : c + 1 < others;
                        const uint64_t vb = vd + static_cast<uint64_t>(st_v * (Cfg::kTile >> 4));
                        ok = ok && wait(&sm.p_full[s][0], phase);
                        if (ok && turns_now) ok = wait(&sm.turn[s], turns++ & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int h2 = 0; h2 < NK / 64; ++h2) {  // O_s += P_s V, the second 64 keys as soon as their weights are there
                            if (h2 == 1) {
                                ok = wait(&sm.p_full[s][1], phase);
                                if (!ok) break;
                                tc_fence_after();
                            }
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
#pragma unroll
                                for (int i = 4 * h2; i < 4 * h2 + 4; ++i)
                                    dp_mma_ts(tmem + 256 + s * 128, tmem + s * 128 + part * (NK / 2) + i * 8,
                                              vb + static_cast<uint64_t>(i * 2048 >> 4), idesc_o,
                                              !(c % kDpRun<kParts> == 0 && part == 0 && i == 0));
                        }
                        if (!ok) break;
                        if (next) {
                            scores(st_k, c + 2 == count, pass);
                        } else {
                            if (pass) mbar_arrive(&sm.turn[s ^ 1]);
                            tc_commit(&sm.o_full[s]);
                        }
                        tc_commit(&sm.empty[st_v]);
                    }
                    if constexpr (!kAlt) {  // tiles that only the other stage needs
                        for (int j = 2 * count; ok && j < 2 * w.total; ++j) {
                            ok = landed();
                            if (ok) mbar_arrive(&sm.empty[bar]);
                            pass_copy();
                        }
                    }
                    slots += 2 * w.total;
                    tiles += count;
                    if (ok) mbar_arrive(&sm.item_done);
                }
                if (issued) {  // every matrix instruction done before tensor memory is given back
                    tc_commit(&sm.drain[s]);
                    wait(&sm.drain[s], 0);
                }
            }
        }
    } else {
        // 168 x 384 registers at launch: 208 x 256 + 88 x 128 (fp32 outputs, 512 rows at 32,768: 965 us; with 200 and 104
        // 1,001, the groups spill; with 232 and 40 1,069, the copying warps do)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---------------- softmax group s: thread = row of M tile s
        const int s = warp >> 2, m = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // (32 (warp % 4)) << 16
        const uint32_t s_addr = tmem + s * 128 + lanes, o_addr = tmem + 256 + s * 128 + lanes;
        int tiles = 0, tiles_before = 0, done = 0;  // running: the stage's tiles, the items' key tiles, items the stage had tiles of
        bool alive = true;
        for (int k = 0; alive; ++k) {
            DpItem item;
            alive = __all_sync(0xffffffffu, next_item(k, item));
            if constexpr (kAlt) alive = dp_sync_and(alive);  // (the groups meet in the epilogue: both come, or neither)
            if (!alive) break;
            if (item.b < 0) break;
            const DpWork w = dp_work<kAlt, NK>(128 / a.G, item);
            const int h = item.h;
            const int pos = w.L - w.n + min(w.i0 + (kAlt ? 0 : s * w.P) + m / a.G, w.n - 1);
            // the tile's earliest position: key tiles up to it hide nothing
            const int early = w.L - w.n + min(w.i0 + (kAlt ? 0 : s * w.P), w.n - 1);
            const int count = s == 0 ? w.count[0] : w.count[1];
            float row_f = a.scale_log2;  // factor from the row's products to the log2 domain
            if constexpr (kF16 || kAlt) alive = __all_sync(0xffffffffu, wait(&sm.q_full, k & 1));
            if constexpr (kF16) {
                // the row's queries to f16: its largest value into [2^8, 2^9)
                if (!alive) break;
                uint8_t* row = sm.q[s] + m * 128;
                auto chunk = [&](int c) { return reinterpret_cast<uint4*>(row + (c >> 3) * (kDpQBytes / 2) + (((c & 7) ^ (m & 7)) << 4)); };
                uint32_t big = 0;  // largest magnitude as bits
#pragma unroll 4
                for (int c = 0; c < 16; ++c) {
                    const uint4 v = *chunk(c);
                    const uint32_t qw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) big = max(big, max((qw[e] << 16) & 0x7fff0000u, qw[e] & 0x7fff0000u));
                }
                const uint32_t ex = min(max(big >> 23, 9u), 253u);
                const float up = __uint_as_float((262u - ex) << 23);  // 2^(8 - exponent)
                row_f *= __uint_as_float((ex - 8u) << 23);
#pragma unroll 4
                for (int c = 0; c < 16; ++c) {
                    const uint4 v = *chunk(c);
                    *chunk(c) = make_uint4(dp_pack_f16(bf16_lo(v.x) * up, bf16_hi(v.x) * up), dp_pack_f16(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                                           dp_pack_f16(bf16_lo(v.z) * up, bf16_hi(v.z) * up), dp_pack_f16(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.q_turned[s]);
            }
            // f16 form: factors (products, value sums) of the key tile's blocks, loaded a tile ahead; the power of two that
            // O is kept in units of (not below any value block's so far)
            const float2* fac = kF16 ? a.wide_fac + (static_cast<int64_t>(h) * a.cache_tokens + a.cache.starts[w.b]) / kBlock : nullptr;
            float2 fac_now[2], fac_next[2];
            auto load_fac = [&](int c, float2 (&x)[2]) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int blk = 2 * (w.first + c) + y;
                    x[y] = blk * kBlock < w.L ? fac[blk] : make_float2(0.f, 0.f);
                }
            };
            if constexpr (kF16) load_fac(0, fac_next);
            int vexp = 0;  // its exponent, biased (the factors are powers of two, 2^-118 .. 2^119; 0: none yet)
            auto power = [](int e) { return e < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + e) << 23); };  // 2^e, e < 128
            bool coarse = false;  // some block's values were 2^-12 or less of another's: small weights may have lost bits
            constexpr float kLift = kF16 ? 6.f : 0.f;  // f16 weights: at most 2^(6 + 8)
            float top = -INFINITY, sum = 0.f;  // maximum in use (log2 domain), sum of weights
            float acc[kParts > 1 ? kHeadDim : 1];  // fp32 outputs: O of the row
            if constexpr (kParts > 1) {
#pragma unroll
                for (int k = 0; k < kHeadDim; ++k) acc[k] = 0.f;
            }
            auto rescale = [&](float r) {  // O in tensor memory times r
#pragma unroll 1
                for (int q = 0; q < kHeadDim / 32; ++q) {
                    float y[32];
                    dp_ld32(o_addr + 32 * q, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k) y[k] *= r;
                    dp_st32(o_addr + 32 * q, reinterpret_cast<const uint32_t*>(y));
                }
            };
            auto collect = [&]() {  // adds the last two tiles' product to it
                if constexpr (kParts > 1) {
#pragma unroll
                    for (int q = 0; q < kHeadDim / 16; ++q) {
                        uint32_t y[16];
                        tmem_ld16(o_addr + 16 * q, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) acc[16 * q + k] += __uint_as_float(y[k]);
                    }
                }
            };
            auto aside = [&](bool first, bool back) {
                if constexpr (kF16) dp_aside(a.aside, o_addr, top, vexp, first, back);
                else dp_aside_call(a.aside, o_addr, top, vexp, first, back);
            };
            for (int c = 0; alive && c < count; ++c) {
                const int j = kAlt ? 2 * c + s : c, t0 = (w.first + j) * NK;
                alive = __all_sync(0xffffffffu, wait(&sm.s_full[s], (tiles + c) & 1));
                if (!alive) break;
                tc_fence_after();
                if constexpr (kParts > 1) {
                    if (c > 0 && c % kDpRun<kParts> == 0) collect();
                } else {
                    if (c > 0 && c % kDpRun<kParts> == 0) aside(c == kDpRun<kParts>, false);
                }
                if constexpr (kParts > 1) {  // ---- fp32 outputs: 32 scores at a time, O in registers (the code below has no room for it)
                    const bool edge = t0 + NK > early + 1;  // some key is hidden from some row of the tile
                    const int e = (tiles_before + j) % kDpScaleSlots;
                    if constexpr (kWide) {
                        alive = __all_sync(0xffffffffu, wait(&sm.sc_full[e], ((tiles_before + j) / kDpScaleSlots) & 1));
                        if (!alive) break;
                    }
                    // the scores of keys 32 q .. of the tile in the log2 domain (f: what is left to multiply by)
                    const float f = kWide || edge ? 1.f : a.scale_log2;
                    auto scores_of = [&](int q, float (&x)[32]) {
                        dp_ld32(s_addr + kSAt + 32 * q, x);
                        tmem_ld_wait();
                        if constexpr (kWide) {
#pragma unroll
                            for (int k = 0; k < 32; k += 4) {
                                const float4 ks = *reinterpret_cast<const float4*>(&sm.sc[e][0][32 * q + k]);
                                x[k] *= ks.x * a.scale_log2;
                                x[k + 1] *= ks.y * a.scale_log2;
                                x[k + 2] *= ks.z * a.scale_log2;
                                x[k + 3] *= ks.w * a.scale_log2;
                            }
                        }
                        if (edge) {
                            const int seen = pos + 1 - t0 - 32 * q;
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] = k < seen ? (kWide ? x[k] : x[k] * a.scale_log2) : -INFINITY;
                        }
                    };
                    float now = -INFINITY;
                    if (kWide || edge) {
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {
                            float x[32];
                            scores_of(q, x);
#pragma unroll
                            for (int k = 0; k < 32; ++k) now = fmaxf(now, x[k]);
                        }
                    } else {
                        tmem_ld_max64(s_addr + kSAt, now);
                        tmem_ld_wait();
                        now *= f;
                    }
                    if (c == 0) {
                        top = now;
                    } else if (__any_sync(0xffffffffu, now > top + kDpSlack)) {
                        const float next = now > top + kDpSlack ? now : top;
                        const float r = top == -INFINITY ? (next == -INFINITY ? 1.f : 0.f) : dp_exp2(top - next);
#pragma unroll
                        for (int k = 0; k < kHeadDim; ++k) acc[k] *= r;
                        if (c & 1) rescale(r);
                        sum *= r;
                        top = next;
                    }
                    const float base = top == -INFINITY ? 0.f : top;
                    const float2 ff = make_float2(f, f), nb = make_float2(-base, -base);
                    float2 add = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        float x[32];
                        scores_of(q, x);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 y = __ffma2_rn(make_float2(x[2 * k], x[2 * k + 1]), ff, nb);
                            x[2 * k] = dp_exp2(y.x);
                            x[2 * k + 1] = dp_exp2(y.y);
                            add = __fadd2_rn(add, make_float2(x[2 * k], x[2 * k + 1]));
                        }
                        if constexpr (kWide) {
#pragma unroll
                            for (int k = 0; k < 32; k += 4) {
                                const float4 vs = *reinterpret_cast<const float4*>(&sm.sc[e][1][32 * q + k]);
                                // a hidden key's weight stays 0 whatever its scale is
                                x[k] = edge && x[k] == 0.f ? 0.f : x[k] * vs.x;
                                x[k + 1] = edge && x[k + 1] == 0.f ? 0.f : x[k + 1] * vs.y;
                                x[k + 2] = edge && x[k + 2] == 0.f ? 0.f : x[k + 2] * vs.z;
                                x[k + 3] = edge && x[k + 3] == 0.f ? 0.f : x[k + 3] * vs.w;
                            }
                        }
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            uint32_t pk[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                pk[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
                                if (part + 1 < kParts) {
                                    x[2 * k] -= bf16_lo(pk[k]);
                                    x[2 * k + 1] -= bf16_hi(pk[k]);
                                }
                            }
                            dp_st16(s_addr + part * 32 + 16 * q, pk);
                        }
                    }
                    sum += add.x + add.y;
                    dp_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.p_full[s][0]);
                        if constexpr (kWide) mbar_arrive(&sm.sc_empty[e]);
                    }
                    continue;
                } else {
                float x[NK], big[NK / 64];
#pragma unroll
                for (int q = 0; q < NK / 64; ++q) dp_ld64_max(s_addr + 64 * q, x + 64 * q, big[q]);
                float f = row_f;  // x f is the score in the log2 domain (f16 form: times the block's factor)
                if constexpr (kF16) {
                    fac_now[0] = fac_next[0];
                    fac_now[1] = fac_next[1];
                    if (c + 1 < count) load_fac(c + 1, fac_next);
                }
                tmem_ld_wait();
                const bool edge = t0 + NK > early + 1;  // some key is hidden from some row of the tile
                if (edge) {
                    const int seen = pos + 1 - t0;
                    if constexpr (kF16) {
#pragma unroll
                        for (int k = 0; k < NK; ++k) x[k] = k < seen ? x[k] * (f * fac_now[k >> 6].x) : -INFINITY;
                        fac_now[0].x = fac_now[1].x = 1.f;
                    } else {
#pragma unroll
                        for (int k = 0; k < NK; ++k) x[k] = k < seen ? x[k] * f : -INFINITY;
                    }
                    f = 1.f;
                }
                float now;
                if (edge) {  // the scores are not those that the load took the maximum of
                    float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < NK; k += 8)
#pragma unroll
                        for (int z = 0; z < 4; ++z) y[z] = fmaxf(y[z], fmaxf(x[k + z], x[k + 4 + z]));
                    now = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * f;
                } else if constexpr (kF16) {
                    now = fmaxf(big[0] * fac_now[0].x, big[NK / 64 - 1] * fac_now[1].x) * f;
                } else {
                    now = (NK == 128 ? fmaxf(big[0], big[NK / 64 - 1]) : big[0]) * f;
                }
                int vnew = vexp, vblock[2] = {0, 0};
                if constexpr (kF16) {  // the same for every row
                    vblock[0] = static_cast<int>(__float_as_uint(fac_now[0].y) >> 23);
                    vblock[1] = static_cast<int>(__float_as_uint(fac_now[1].y) >> 23);
                    vnew = max(vexp, max(vblock[0], vblock[1]));
                }
                if (c == 0) {
                    top = now;
                } else if (__any_sync(0xffffffffu, now > top + kDpSlack) || (kF16 && vnew > vexp)) {
                    // the maximum grew: the warp's rows of O in tensor memory (no product runs on it now: S of this tile
                    // was computed after the last one) and their sums move to the new one
                    const float next = now > top + kDpSlack ? now : top;
                    const float r = top == -INFINITY ? (next == -INFINITY ? 1.f : 0.f) : dp_exp2(top - next);
                    const float ro = kF16 ? r * power(vexp - vnew) : r;
                    if constexpr (kF16) coarse |= vexp - vnew < -12;
                    rescale(ro);
                    sum *= r;
                    top = next;
                }
                if constexpr (kF16) vexp = vnew;
                const float base = top == -INFINITY ? 0.f : top;
                float2 ff = make_float2(f, f), nb = make_float2(-base, -base);
                float back[2] = {1.f, 1.f};  // f16 form: from a block's weights, in units of its values, to plain ones
                float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h2 = 0; h2 < NK / 64; ++h2) {  // 64 keys at a time: the products with them start while the next are made
                    int unit = 0;  // f16 form: the block's value factor over the one that O is kept in, log2 (at most 0)
                    bool folded = true;
                    if constexpr (kF16) {
                        // weight 2^(x - base + 6) times 2^unit: an exponent's addition, and taken out of the sum again, unless it
                        // is too small for that (a block of tiny scales; the same for the whole CTA)
                        if (vblock[h2] > 0) unit = vblock[h2] - vexp;
                        folded = unit >= -60;
                        coarse |= unit < -12;
                        const float up = kLift + (folded ? static_cast<float>(unit) : 0.f);
                        ff = make_float2(f * fac_now[h2].x, f * fac_now[h2].x);
                        nb = make_float2(up - base, up - base);
                        back[h2] = folded ? power(-unit) : 1.f;
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float* z = x + 64 * h2 + 32 * q;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 y = __ffma2_rn(make_float2(z[2 * k], z[2 * k + 1]), ff, nb);
                            z[2 * k] = dp_exp2(y.x);
                            z[2 * k + 1] = dp_exp2(y.y);
                            add[kF16 ? h2 : k & 1] = __fadd2_rn(add[kF16 ? h2 : k & 1], make_float2(z[2 * k], z[2 * k + 1]));
                        }
                        if (kF16 && !folded) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) z[k] *= power(unit);
                        }
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            pk[k] = kF16 ? dp_pack_f16(z[2 * k], z[2 * k + 1]) : pack_bf16x2(z[2 * k], z[2 * k + 1]);
                        dp_st16(s_addr + 32 * h2 + 16 * q, pk);
                    }
                    dp_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[s][h2]);
                }
                sum += (add[0].x + add[0].y) * back[0] + (add[1].x + add[1].y) * back[1];
                }
            }
            // (the item is read again here, so that the loop over its tiles need not keep it in registers)
            {
                const DpItem item = sm.info[k % kDpInfo];
                const DpWork w = dp_work<kAlt, NK>(128 / a.G, item);
                const int h = item.h, count = s == 0 ? w.count[0] : w.count[1];
                const int i = w.i0 + (kAlt ? 0 : s * w.P) + m / a.G, g = m % a.G;
                const bool mine = m < w.P * a.G && i < w.n;
                const int pos = w.L - w.n + min(i, w.n - 1);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.info_empty[k % kDpInfo]);
                if constexpr (kWide) {  // scales of tiles that only the other group needs
                    for (int j = tiles_before + count; alive && j < tiles_before + w.total; ++j) {
                        alive = __all_sync(0xffffffffu, wait(&sm.sc_full[j % kDpScaleSlots], (j / kDpScaleSlots) & 1));
                        if (alive && lane == 0) mbar_arrive(&sm.sc_empty[j % kDpScaleSlots]);
                    }
                }
                // ---------------- epilogue
                bool have = count > 0;
                if (alive && have) alive = __all_sync(0xffffffffu, wait(&sm.o_full[s], done++ & 1));
                tc_fence_after();
                if (alive && have) collect();
                if constexpr (kParts == 1) {
                    if (alive && count > kDpRun<kParts>) aside(false, true);
                }
                constexpr int kRun = 32;  // values of the row that are finished at a time
                auto row_of_o = [&](int q, float (&y)[kRun]) {
                    if constexpr (kParts > 1) {
#pragma unroll
                        for (int k = 0; k < kRun; ++k) y[k] = acc[kRun * q + k];
                    } else {
                        dp_ld32(o_addr + kRun * q, y);
                        tmem_ld_wait();
                    }
                };
                float f0 = 1.f, f1 = 0.f;
                float* other = reinterpret_cast<float*>(&sm.q[0][0]);  // [128 dims][128 rows]
                if constexpr (kAlt) {
                    // the second stream's state goes through the query buffers, once both streams' products are done (where a wait
                    // gave up, all 256 threads stop here together)
                    alive = dp_sync_and(alive);
                    if (!alive) break;
                    if (s == 1 && have) {
#pragma unroll(kParts > 1 ? 4 : 1)
                        for (int q = 0; q < kHeadDim / kRun; ++q) {
                            float y[kRun];
                            row_of_o(q, y);
#pragma unroll
                            for (int k = 0; k < kRun; ++k) other[(kRun * q + k) * 128 + m] = y[k];
                        }
                    }
                    if (s == 1) sm.other_ml[m] = make_float2(have ? top : -INFINITY, have ? sum : 0.f);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the next item's queries land here)
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                    if (s == 0 && w.count[1] > 0) {
                        const float2 ml = sm.other_ml[m];
                        const float t2 = fmaxf(top, ml.x);
                        f0 = top == -INFINITY ? 0.f : dp_exp2(top - t2);
                        f1 = ml.x == -INFINITY ? 0.f : dp_exp2(ml.x - t2);
                        sum = sum * f0 + ml.y * f1;
                        top = t2;
                    }
                }
                const bool split_up = item.nsplit > 1;
                if (alive && (have || split_up) && !(kAlt && s == 1)) {  // (kAlt: group 0 writes)
                    constexpr int kRows = kAlt ? 128 : 256;  // rows of an item's part
                    const int64_t q_row = (static_cast<int64_t>(w.c0 + min(i, w.n - 1)) * a.H + h) * a.G + g;
                    const int64_t part_row = static_cast<int64_t>(item.part) * kRows + s * 128 + m;
                    float most = 0.f;  // f16 form: the row's largest value, in units of w x V16
                    bool spoiled = false;  // some value of the row is not finite
                    const float vref = kF16 ? __uint_as_float(static_cast<uint32_t>(vexp) << 23) : 1.f;
                    const float inv = kF16 ? vref / sum : 1.f / sum;  // (parts: O in plain units, as their join expects)
                    if (have) {
                        const float to = split_up ? (kF16 ? vref : 1.f) : inv;
#pragma unroll(kParts > 1 ? 4 : 1)
                        for (int q = 0; q < kHeadDim / kRun; ++q) {
                            float y[kRun];
                            row_of_o(q, y);
                            if constexpr (kAlt) {
                                if (w.count[1] > 0) {
#pragma unroll
                                    for (int k = 0; k < kRun; ++k) y[k] = y[k] * f0 + other[(kRun * q + k) * 128 + m] * f1;
                                }
                            }
                            float2 zero[4] = {};  // 0 unless a value is infinite or NaN
#pragma unroll
                            for (int k = 0; k < kRun; k += 8)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    zero[e] = __ffma2_rn(make_float2(y[k + 2 * e], y[k + 2 * e + 1]), make_float2(0.f, 0.f), zero[e]);
                            spoiled |= !(((zero[0].x + zero[0].y) + (zero[1].x + zero[1].y)) + ((zero[2].x + zero[2].y) + (zero[3].x + zero[3].y)) == 0.f);
                            if constexpr (kF16) {
                                float big[4] = {most, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int k = 0; k < kRun; ++k) big[k & 3] = fmaxf(big[k & 3], fabsf(y[k]));
                                most = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
                            }
#pragma unroll
                            for (int k = 0; k < kRun; k += 2) {
                                const float2 z = __fmul2_rn(make_float2(y[k], y[k + 1]), make_float2(to, to));
                                y[k] = z.x;
                                y[k + 1] = z.y;
                            }
                            if (!mine) {
                                // (a row of the tile that no query has)
                            } else if (split_up || !a.out_bf16) {
                                float* to_row = split_up ? a.part_o + part_row * kHeadDim : static_cast<float*>(a.out) + q_row * kHeadDim;
                                float4* dst = reinterpret_cast<float4*>(to_row + kRun * q);
#pragma unroll
                                for (int k = 0; k < kRun / 4; ++k) dst[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                            } else {
                                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + q_row * kHeadDim + kRun * q);
#pragma unroll
                                for (int k = 0; k < kRun / 8; ++k)
                                    dst[k] = make_uint4(pack_bf16x2(y[8 * k], y[8 * k + 1]), pack_bf16x2(y[8 * k + 2], y[8 * k + 3]),
                                                        pack_bf16x2(y[8 * k + 4], y[8 * k + 5]), pack_bf16x2(y[8 * k + 6], y[8 * k + 7]));
                            }
                            __syncwarp();  // the next load is the whole warp's
                        }
                    }
                    if (split_up && mine) *reinterpret_cast<float2*>(a.part_ml + part_row * 2) = make_float2(top, sum);
                    if constexpr (!kWide) {  // (bf16 integers are finite, and a hidden key's weight ignores its scale)
                        const int keys = (w.first + (kAlt ? w.total : count)) * NK, end = min(pos + 1, keys);
                        // only a value past the row's position makes a row wrong that is not finite (the row's own keys and
                        // values give what the formula gives, and a sum that is not finite is theirs)
                        spoiled = spoiled && mine && have && fabsf(sum) < INFINITY;
                        if (__any_sync(0xffffffffu, spoiled)) {
                            const int least = static_cast<int>(__reduce_min_sync(0xffffffffu, mine ? static_cast<uint32_t>(pos) : 0x7fffffffu));
                            const int bad = dp_last_bad(a, w.b, h, max(least + 1, w.first * NK), min(keys, w.L));  // (every lane)
                            spoiled = spoiled && bad > pos;
                        }
                        // f16 form: a row that lives on blocks whose values are tiny (2^-12) beside another block's (even one
                        // that it does not see) has small weights there, off by up to 2^-25 each, L^1/2 2^-12 in units where
                        // it has 2^10 or more when nothing was lost.  Further apart (2^-22), or where keys or values of a
                        // block have lost bits to another's of the block, they may be all that a row sees (or that one of its
                        // values has: codes of 0 in the large ones), so every row of the tile is computed again.
                        if constexpr (kF16) {
                            if (coarse || sm.lost) {
                                const int apart = dp_apart(fac, 2 * w.first, min(2 * (w.first + count), (w.L + kBlock - 1) / kBlock));
                                if (apart > 22 || (apart > 12 && most < 1024.f)) spoiled = fabsf(sum) < INFINITY;
                            }
                        }
                        uint32_t again = __ballot_sync(0xffffffffu, mine && spoiled && have);
                        while (again) {  // these rows once more, by the whole warp
                            DpAgain x;
                            int64_t pr[kDpAgain];
#pragma unroll
                            for (int r = 0; r < kDpAgain; ++r) {  // (the last of them several times where there are fewer)
                                const int from = __ffs(again) - 1;
                                if (r == kDpAgain - 1 || (again & (again - 1)) != 0) again &= again - 1;
                                x.q_row[r] = __shfl_sync(0xffffffffu, q_row, from);
                                pr[r] = __shfl_sync(0xffffffffu, part_row, from);
                                x.end[r] = __shfl_sync(0xffffffffu, end, from);
                            }
                            dp_rows_again<kF16>(a, w.b, h, w.first * NK, x);
#pragma unroll
                            for (int r = 0; r < kDpAgain; ++r) {
                                const float* y = x.o[r];
                                const int64_t at = x.q_row[r] * kHeadDim + 4 * lane;
                                const float f = 1.f / x.l[r];
                                if (split_up) {  // (in the units of the other parts' sums)
                                    constexpr float kUnits = kF16 ? 64.f : 1.f;
                                    *reinterpret_cast<float4*>(a.part_o + pr[r] * kHeadDim + 4 * lane) =
                                        make_float4(y[0] * kUnits, y[1] * kUnits, y[2] * kUnits, y[3] * kUnits);
                                    if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + pr[r] * 2) = make_float2(x.m[r], x.l[r] * kUnits);
                                } else if (a.out_bf16) {
                                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                                        make_uint2(pack_bf16x2(y[0] * f, y[1] * f), pack_bf16x2(y[2] * f, y[3] * f));
                                } else {
                                    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
                                }
                            }
                        }
                    }
                }
                if constexpr (kAlt) {
                    if (s == 0) {  // the query buffers are free again
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.q_empty);
                    }
                }
                tc_fence_before();
                tiles += count;
                tiles_before += w.total;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of split items: CTA x takes split item x, a warp every 4 gridDim.y-th of its rows, 4 of the 128
// values a lane, eight parts' loads in flight: a running maximum m and sum of 2^(m_i - m) O_i in the parts' order, the
// same every time.
constexpr int kDjThreads = 128;
template <bool kAlt>
__global__ void __launch_bounds__(kDjThreads, 8) dense_join_kernel(const DenseArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kRows = kAlt ? 128 : 256;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int2 head = *a.split_head;  // split items, parts of each
    const int4 it = a.split_items[blockIdx.x];
    const uint32_t err = *a.err;
    // (where a wait gave up, an item may have been left that nobody wrote down)
    if (static_cast<int>(blockIdx.x) >= head.x || (err & kErrWaitTimeout)) return;
    const int nsplit = head.y, h = it.z;
    const int c0 = a.cu_rows[it.x], n = a.cu_rows[it.x + 1] - c0, P = 128 / a.G, i0 = it.y * P * (kAlt ? 1 : 2);
    const int64_t base = static_cast<int64_t>(blockIdx.x) * nsplit * kRows;
    for (int x = blockIdx.y * 4 + warp; x < kRows; x += gridDim.y * 4) {
        const int s = x >> 7, m0 = x & 127, i = i0 + s * P + m0 / a.G, g = m0 % a.G;
        if (m0 >= P * a.G || i >= n) continue;
        float m = -INFINITY, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int y0 = 0; y0 < nsplit; y0 += 8) {
            float4 p[8];
            float2 ml[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t row = base + static_cast<int64_t>(y0 + u) * kRows + x;
                ml[u] = make_float2(-INFINITY, 0.f);
                if (y0 + u < nsplit) {
                    ml[u] = *reinterpret_cast<const float2*>(a.part_ml + row * 2);
                    p[u] = *reinterpret_cast<const float4*>(a.part_o + row * kHeadDim + 4 * lane);
                }
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < 8; ++u) top = fmaxf(top, ml[u].x);
            if (m != -INFINITY) {
                const float f = dp_exp2(m - top);
                l *= f;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= f;
            }
            m = top;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (y0 + u >= nsplit) break;
                // a part without keys (maximum -inf) weighs nothing, unless its sum is NaN
                const float w = ml[u].x == -INFINITY ? (ml[u].y == ml[u].y ? 0.f : ml[u].y) : dp_exp2(ml[u].x - m);
                if (w != 0.f) {
                    l = fmaf(w, ml[u].y, l);
                    v[0] = fmaf(w, p[u].x, v[0]);
                    v[1] = fmaf(w, p[u].y, v[1]);
                    v[2] = fmaf(w, p[u].z, v[2]);
                    v[3] = fmaf(w, p[u].w, v[3]);
                }
            }
        }
        const float inv = 1.f / l;
        const int64_t out = (((static_cast<int64_t>(c0 + i) * a.H + h) * a.G) + g) * kHeadDim + 4 * lane;
        if (a.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out) =
                make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + out) =
                make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    }
}

template <int kParts, int kForm, bool kAlt>
static cudaError_t launch_dense_prompt(DenseArgs a, int items, cudaStream_t stream) {
    auto* kernel = dense_prompt_kernel<kParts, kForm, kAlt>;
    const size_t smem = sizeof(DpSmem<kParts, kForm>) + 1024;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    a.places = std::min(device_sm_count(), kDenseMaxShares);
    a.wait_ns = kWaitLimitNs + kDpAgainNs * static_cast<uint64_t>(a.max_cache_len);
    // every item, and room for the parts of the last wave's: what the rule would choose for the host's counts where
    // there is one sequence (or window each), which they tell exactly, else two a place.  (3 sequences of 64 rows at
    // 32,768, one head: 78 us, without parts 347; 8 packed prompts of up to 2,047, which have nothing to split: 101, and
    // 97 without the launch that finds that out; one and four a place are as two.)
    const int64_t whole = static_cast<int64_t>(items) * a.H;
    const float tiles = a.max_cache_len / 128.f;
    const int rest = static_cast<int>(whole % a.places);
    a.parts_most = 0;
    if (kAlt || a.num_seqs == 1) {
        int best = 1;
        for (int n = 2; n <= 32 && rest * n <= kDenseMaxParts && tiles >= 4.f * n; ++n)
            if (dp_cost(rest, a.places, tiles, n) < dp_cost(rest, a.places, tiles, best)) best = n;
        if (best > 1) a.parts_most = rest * best;
    } else if (tiles >= 8.f) {
        a.parts_most = 2 * a.places;
    }
    const int64_t grid = std::min<int64_t>(whole + a.parts_most, a.places);
    kernel<<<static_cast<unsigned>(grid), kDpThreads, smem, stream>>>(*a.q_map, *a.k_map, *a.v_map, a, items);
    if ((e = cudaGetLastError()) != cudaSuccess || a.parts_most == 0) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(items) * a.H, a.places)), kAlt ? 16 : 8, 1);
    cfg.blockDim = dim3(kDjThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dense_join_kernel<kAlt>, a);
}

cudaError_t run_dense_prompt(const DenseArgs& a, int items, cudaStream_t stream) {
    if (a.kv_int8)
        return a.out_bf16 ? launch_dense_prompt<1, kDpF16, false>(a, items, stream)
                          : launch_dense_prompt<3, kDpInt, false>(a, items, stream);
    return a.out_bf16 ? launch_dense_prompt<1, kDpBf16, false>(a, items, stream)
                      : launch_dense_prompt<3, kDpBf16, false>(a, items, stream);
}

cudaError_t run_dense_window(const DenseArgs& a, int items, cudaStream_t stream) {
    return a.out_bf16 ? launch_dense_prompt<1, kDpBf16, true>(a, items, stream)
                      : launch_dense_prompt<3, kDpBf16, true>(a, items, stream);
}

}  // namespace msa
