// Attention over every cached position for decode rows and drafted windows (1 to 8 rows a sequence) of a batch in which
// groups of sequences share a prefix: the prefix is read once for all rows of the group.
//   out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m),  x_t = scale log2(e) q.k_t over t <= p
// A softmax over a set of keys splits into parts (O, m, l: unnormalised sum, maximum, sum of weights) over any division
// of the keys, joined by weights 2^(m_i - m).  Here the keys of a row are divided into
//   the group's shared positions [0, S)     one item for up to 2 x 128 (row, head) pairs of the group and a KV head
//   the sequence's own positions [S, L - n) one item for the sequence's (row, head) pairs and a KV head
//   the n rows' own positions [L - n, p]    at most 8 keys, in fp32 by the kernel that joins the parts
// so that the first two have no causal edge: every row of an item sees every key of it, and no value of a later token is
// ever multiplied with.
//
// dense_shared_kernel.  An item is an M tile of 128 rows (row = neighbouring query rows x G heads; a sequence's n G rows
// leave the others of the tile empty) or two of them, and its keys in tiles of NK:
//   S[128, NK] = Q K^T     operands from shared memory (TMA, 128-byte swizzle), S in tensor memory
//   P = 2^(x - m)          a thread a row, written over S (m is raised only where it would grow by more than 8)
//   O[128, 128] += P V     P from tensor memory, V as it lies
// Two stages of 128 columns of S and of O: two M tiles that take turns on the tensor pipe, or one M tile whose stages
// take alternate key tiles (the first of an item in turn: items of one tile keep both busy).  One CTA per SM; all items'
// key tiles lie on a line, item after item, that is cut into even shares; a CTA's shares of items leave their parts in the
// workspace.  On the line a tile of two M tiles is half as long again as one of a single M tile (1.55 us for 1.0 to 1.4
// measured), and going on to another item counts for one and a half tiles (tiles of equal length: 3% slower at 256
// sequences, 11% with several groups; one or two tiles an item: up to 4% slower).
// The next item is walked to, not divided out: those loads and divisions stood before the copies of a short item (1 to 2 us).
// Values past the end of a sequence become zero by the softmax warps, as the copying warp cannot go on while it waits for
// them.  Both together: 157 for 168 us at 256 sequences of one to four tiles.
//
// int8 caches.  The tiles land as codes, and four more warps write them as bf16, exactly (7 instructions for 4), into the
// ring that the products read; a key's scale multiplies its scores and a value's the weights, after their sum.  The codes
// of a tile become bf16 once for all rows of an item.  A thread's 128 scores take 64 products and no reducing load then:
// 2.9 us a tile of two M tiles for 1.55; the scales are loaded 32 at a time (one by one as used: 64 for 60 us).
//
// dense_shared_join.  A CTA takes a row and a KV head: the row's own keys, then the parts, whose places follow from the
// same line by arithmetic (slot = item + CTA, which is different for every pair of them that meets, as both ascend along
// the line).  Parts lie [dim / 4][row][4], so that the rows of a tile are stored and loaded in whole lines.
//
// Numerics.  bf16 outputs: weights as one bf16 (2^-8 at most, at random), as prompt chunks have them and decode rows without
// groups have not (two parts; int8 caches: f16).  Two parts here are 71 us for 57 at 32 sequences over an int8 cache, whose
// error against the formula they lower from 2.4e-3 to 1.7e-3 in the norm, the output's own rounding (a cached value is off by
// up to 1/254 of its head's largest).  At most 32,768 keys to a sum in tensor memory (longer ones are added up in the CTA's
// part), as the tensor cores cut what an addition loses instead of rounding it (2^-24 an addition of 16 keys).  fp32 outputs:
// weights as three bf16 parts, NK = 64, O taken from tensor memory every second tile and summed in registers.
//
// Bound by the tensor pipe where many rows share (two M tiles: 1.55 us a tile of 128 keys for 1.3 at the pipe's rate), by
// the chain of one tile's scores, weights and products elsewhere (2.7 us a stage: own positions go at 48 KB a us and SM,
// about HBM's rate over all SMs), and by its beginning: 5 us to the first copy, 7 to 8 to the first scores.
// Measured, whole calls of 4 x 16 heads: 64 sequences behind 32,768 positions and 100 to 2,000 of their own, 81 us (prefix
// once and own positions: 24.6 us of memory, 35.8 of products; without groups 408 us); 256 behind 8,192, 132 us; 8 behind
// 1,984, 18.5 us (17.7); int8, 32 behind 16,384, 57 us (96); 16 behind 8,192 with fp32 outputs, 36.4 us (46).  Where little
// is shared the calls take longer than without groups: 6 us of beginning and join (int8 10), and own positions cost, for what
// they cost there, 1.05 (bf16), 1.5 (fp32 outputs), 2.4 (int8) and 3 times (int8, fp32 outputs).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tensor_rows.cuh"

namespace msa {

// Softmax groups: warps 0-3, 4-7; 8 and 10 copies, 9 and 11 matrix instructions; int8 caches: 12-15 make bf16 of the codes.
constexpr int kDsThreads = 384, kDsThreadsInt8 = 512;
constexpr int kDsQBytes = 128 * kHeadDim * 2;
constexpr int kDsPartKeys = 32768;  // most keys of a sum in tensor memory
// Lengths on the line, in half tiles: a key tile of one M tile, of two, and what an item counts for besides.
constexpr int kDsSingle = 2, kDsPair = 3, kDsExtra = 3;
constexpr int kDsInfo = 4;          // items published ahead
constexpr float kDsSlack = 8.f;     // log2 by which the running maximum may lag

// A CTA's share of an item.
struct DsItem {
    int b;             // sequence whose table is read; < 0: no more items
    int row, rows;     // first query row of the item, query rows of its entry from there on
    int h, key, end;   // KV head; first key of the share; end of the entry's keys
    int tiles, pair;   // key tiles; two M tiles (or one, the stages on alternate key tiles)
    int cap;           // rows of a stage's part
    int more;          // 1: earlier keys of the item are in its parts already
    int64_t part;      // first row of its parts in the workspace
};

template <int kParts, bool kInt8>
struct DsCfg {
    static constexpr int NK = kParts == 1 ? 128 : 64;
    static constexpr int kTile = NK * kHeadDim * 2;  // bytes of a K or V tile
    static constexpr int kStages = (kInt8 ? 3 : 5) * (128 / NK);
    static constexpr int kCodes = 3 * (128 / NK);  // int8: tiles of codes in flight
    // int8: tiles whose scales are kept.  When tile t is converted its slot has been given back by the values of tile t - 2
    // (64-key tiles: t - 4 at the latest), whose softmax is then done.
    static constexpr int kScales = 8;
    static constexpr int kThreads = kInt8 ? kDsThreadsInt8 : kDsThreads;
    static constexpr int kSAt = kParts == 1 ? 0 : 64;  // column of S in its 128 (as in the prompt kernel: P's parts from 0 on)
    static constexpr int kRun = kDsPartKeys / NK;      // most tiles of a sum
};

template <int kParts, bool kInt8>
struct __align__(1024) DsSmem {
    using Cfg = DsCfg<kParts, kInt8>;
    uint8_t q[2][kDsQBytes];
    uint8_t ring[Cfg::kStages][Cfg::kTile];
    uint8_t codes[kInt8 ? Cfg::kCodes : 1][kInt8 ? Cfg::kTile / 2 : 16];
    float sc[kInt8 ? Cfg::kScales : 1][2][kInt8 ? Cfg::NK : 4];  // scales of a tile's keys and values
    uint64_t code_full[Cfg::kCodes], code_empty[Cfg::kCodes];
    // Copies landed: of pairs [0], of the two stages on alternate tiles [1], [2], each counted by itself, so that an issuer
    // sees all phases of the barriers that it waits for.
    uint64_t full[3][Cfg::kStages], empty[Cfg::kStages];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2][2], o_full[2], turn[2], drain[2];  // P: by halves of the key tile
    uint64_t info_full[kDsInfo], info_empty[kDsInfo], item_done[2];
    DsItem info[kDsInfo];
    uint32_t tmem, err;
    int64_t group_parts;  // parts of all groups
    int first;         // the entry where the CTA's share begins, and what is known of it
    SharedEntry first_entry;
    int64_t scan_line[Cfg::kThreads / 32];
    int32_t scan_items[Cfg::kThreads / 32];
};
static_assert(sizeof(DsSmem<1, false>) + 1024 <= 227 * 1024, "shared-prefix attention exceeds 227 KB of shared memory");
static_assert(sizeof(DsSmem<3, false>) + 1024 <= 227 * 1024, "shared-prefix attention (fp32) exceeds 227 KB of shared memory");
static_assert(sizeof(DsSmem<1, true>) + 1024 <= 227 * 1024, "shared-prefix attention (int8) exceeds 227 KB of shared memory");
static_assert(sizeof(DsSmem<3, true>) + 1024 <= 227 * 1024, "shared-prefix attention (int8, fp32) exceeds 227 KB of shared memory");

// Entries of the line: the groups, then the sequences.  The query rows [row, row + rows) see all keys [key, end).
struct DsEntry {
    int b, row, rows, key, end;
};

// The shared positions of group g in whole blocks (0 where its metadata is bad), its sequences and rows.
__device__ __forceinline__ int ds_group(const SharedArgs& a, int g, DsEntry& x, int& last, bool& bad) {
    const int b0 = a.group_starts[g], b1 = a.group_starts[g + 1], S = a.group_shared[g];
    bad = b0 < 0 || b1 < b0 || b1 > a.num_seqs || S < 0 || S > a.max_shared_len;
    if (bad) return 0;
    const int c0 = a.cu_rows[b0], c1 = a.cu_rows[b1];
    bad = c0 < 0 || c1 < c0 || c1 > a.total_rows || c1 - c0 > a.max_group_rows;
    if (bad) return 0;
    x = DsEntry{b0, c0, c1 - c0, 0, S & ~(kBlock - 1)};
    last = b1;
    return x.end;
}

// The shared positions of sequence b, in whole blocks, and its group (-1: none).
__device__ __forceinline__ int ds_shared_of(const SharedArgs& a, int b, int& g) {
    int lo = 0, hi = a.num_groups;  // largest group that begins at or before b
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.group_starts[mid] <= b) lo = mid; else hi = mid;
    }
    g = -1;
    DsEntry x;
    int last;
    bool bad;
    const int S = ds_group(a, lo, x, last, bad);
    if (bad || b < x.b || b >= last || S == 0) return 0;
    g = lo;
    return S;
}

// Sequence b; rows = 0: it has none, or its metadata is bad.
__device__ __forceinline__ DsEntry ds_seq(const SharedArgs& a, int b, int& g, bool& bad) {
    const int c0 = a.cu_rows[b], n = a.cu_rows[b + 1] - c0, L = a.cache_lens[b];
    const int S = ds_shared_of(a, b, g);
    bad = n < 0 || n > min(a.max_rows_per_seq, kDecodeMaxRows) || c0 < 0 || c0 + n > a.total_rows || L < n || L > a.max_cache_len ||
          L - n < S;
    if (n == 0) bad = false;
    if (bad || n == 0) return DsEntry{b, 0, 0, 0, 0};
    return DsEntry{b, c0, n, S, L - n};
}

// How an entry lies on the line: `units` items a head (of up to two M tiles), each `chunks` pieces of up to `run` tiles.
struct DsSize {
    int tiles, chunks, units, unit, w;  // key tiles; pieces they make; items a head; an item's length on the line, a tile's
};
__device__ __forceinline__ DsSize ds_size(const SharedArgs& a, const DsEntry& x, int NK) {
    DsSize s{};
    if (x.rows == 0 || x.end <= x.key) return s;
    const int run = kDsPartKeys / NK, P = 128 / a.G, mt = x.rows <= P ? 1 : (x.rows + P - 1) / P;
    s.tiles = (x.end - x.key + NK - 1) / NK;
    s.chunks = (s.tiles + run - 1) / run;
    s.units = (mt + 1) / 2;
    s.w = mt > 1 ? kDsPair : kDsSingle;
    s.unit = s.tiles * s.w + s.chunks * kDsExtra;
    return s;
}
__device__ __forceinline__ DsEntry ds_entry(const SharedArgs& a, int e, bool& bad) {
    if (e >= a.num_groups) {
        int g;
        return ds_seq(a, e - a.num_groups, g, bad);
    }
    DsEntry x{};
    int last;
    ds_group(a, e, x, last, bad);
    return x;
}

// Tiles of a piece that begin before x on the line from its first tile on.
__device__ __forceinline__ int ds_tiles_before(int x, int w) {
    return x <= 0 ? 0 : (w == kDsPair ? (x + kDsPair - 1) / kDsPair : (x + kDsSingle - 1) / kDsSingle);
}

// CTAs that share a line, and where share c begins (the largest c whose share begins at or before a place: ds_owner).
__device__ __forceinline__ int ds_shares(int64_t line, int grid) {
    const int64_t n = line / (kDsExtra + 2 * kDsPair);  // (no share is then without a tile of an item that goes through it)
    return static_cast<int>(n < 1 ? 1 : (n < grid ? n : grid));
}
__device__ __forceinline__ int64_t ds_cut(int64_t line, int c, int shares) { return line * c / shares; }
__device__ __forceinline__ int ds_owner(int64_t line, int64_t at, int shares) {
    return static_cast<int>(((at + 1) * shares - 1) / line);
}
__device__ __forceinline__ SharedEntry ds_load(const SharedEntry* p) {
    SharedEntry y;
    reinterpret_cast<int4*>(&y)[0] = reinterpret_cast<const int4*>(p)[0];
    reinterpret_cast<int4*>(&y)[1] = reinterpret_cast<const int4*>(p)[1];
    return y;
}

__device__ __forceinline__ uint4 ds_ld_shared(uint32_t at) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
    return w;
}
// x[i] times the 32 floats at `at` (the loads first: one behind another they would each take their latency).
__device__ __forceinline__ void ds_times32(float* x, uint32_t at) {
    uint4 f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = ds_ld_shared(at + 16 * i);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 y0 = __fmul2_rn(make_float2(x[4 * i], x[4 * i + 1]), make_float2(__uint_as_float(f[i].x), __uint_as_float(f[i].y)));
        const float2 y1 = __fmul2_rn(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(__uint_as_float(f[i].z), __uint_as_float(f[i].w)));
        x[4 * i] = y0.x, x[4 * i + 1] = y0.y, x[4 * i + 2] = y1.x, x[4 * i + 3] = y1.y;
    }
}
__device__ __forceinline__ void ds_st_shared(uint32_t at, uint4 w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}

// A later piece of an item's keys: its O (tensor memory), maximum and sum are added to what this thread has stored of the
// earlier ones, so that parts are as many as items and CTAs, however long the keys.  A piece without a key above -inf says
// nothing, unless its sum is NaN.  By the whole warp.
__device__ __forceinline__ void ds_add_piece(uint32_t o_addr, float4* dst, int cap, float2* ml, bool mine, float top, float sum) {
    const float2 was = mine ? *ml : make_float2(-INFINITY, 0.f);
    const bool before = was.x != -INFINITY || was.y != was.y, now = mine && (top != -INFINITY || sum != sum);
    const float most = fmaxf(was.x, top);
    const float f0 = was.x == -INFINITY ? was.y : dp_exp2(was.x - most), f1 = top == -INFINITY ? sum : dp_exp2(top - most);
#pragma unroll 1
    for (int q = 0; q < kHeadDim / 32; ++q) {
        float y[32];
        dp_ld32(o_addr + 32 * q, y);
        tmem_ld_wait();
        if (before && now) {
            float4 o[8];  // (the loads first: each behind a store would take its latency, 11 us at three groups)
#pragma unroll
            for (int d = 0; d < 8; ++d) o[d] = dst[static_cast<int64_t>(8 * q + d) * cap];
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                y[4 * d] = fmaf(o[d].x, f0, y[4 * d] * f1);
                y[4 * d + 1] = fmaf(o[d].y, f0, y[4 * d + 1] * f1);
                y[4 * d + 2] = fmaf(o[d].z, f0, y[4 * d + 2] * f1);
                y[4 * d + 3] = fmaf(o[d].w, f0, y[4 * d + 3] * f1);
            }
        }
        if (now) {
#pragma unroll
            for (int d = 0; d < 8; ++d)
                dst[static_cast<int64_t>(8 * q + d) * cap] = make_float4(y[4 * d], y[4 * d + 1], y[4 * d + 2], y[4 * d + 3]);
        }
        __syncwarp();  // the next load is the whole warp's
    }
    if (now) *ml = before ? make_float2(most, fmaf(was.y, f0, sum * f1)) : make_float2(top, sum);
}

// Few items have more than one piece: a call where registers are short (fp32 outputs 37.3 us, inline 38.0; int8 57.3 and 58.3;
// 64 sequences in bf16 88.8, inline 79.7).
__device__ __noinline__ void ds_call_add_piece(uint32_t o_addr, float4* dst, int cap, float2* ml, bool mine, float top, float sum) {
    ds_add_piece(o_addr, dst, cap, ml, mine, top, sum);
}

template <int kParts, bool kInt8>
__global__ void __launch_bounds__(kInt8 ? kDsThreadsInt8 : kDsThreads, 1) dense_shared_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                    const __grid_constant__ CUtensorMap k_map,
                                                                    const __grid_constant__ CUtensorMap v_map,
                                                                    const SharedArgs a) {
    using Cfg = DsCfg<kParts, kInt8>;
    using Smem = DsSmem<kParts, kInt8>;
    constexpr int kThreads = Cfg::kThreads, kCodes = Cfg::kCodes;
    constexpr int NK = Cfg::NK, kStages = Cfg::kStages, kHalf = Cfg::kTile / 2, kSAt = Cfg::kSAt, kRun = Cfg::kRun;
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &sm.err); };
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            for (int k = 0; k < 3; ++k) mbar_init(&sm.full[k][s], kInt8 ? 4 : 2);  // two warps copy a half each (int8: four convert)
            mbar_init(&sm.empty[s], 2);                                // both issuers (alternate tiles: one, and the copier for the other)
        }
        for (int s = 0; s < kDsInfo; ++s) {
            mbar_init(&sm.info_full[s], 1);
            mbar_init(&sm.info_empty[s], kInt8 ? 15 : 11);  // a copier, two issuers, eight softmax warps, four that convert
        }
        for (int s = 0; s < kCodes; ++s) {
            mbar_init(&sm.code_full[s], 2);
            mbar_init(&sm.code_empty[s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.item_done[s], 2);
            mbar_init(&sm.q_full[s], 1);
            mbar_init(&sm.q_empty[s], 2);
            mbar_init(&sm.s_full[s], 1);
            mbar_init(&sm.p_full[s][0], 4);
            mbar_init(&sm.p_full[s][1], 4);
            mbar_init(&sm.o_full[s], 1);
            mbar_init(&sm.turn[s], 1);
            mbar_init(&sm.drain[s], 1);
        }
        sm.err = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane < 3) prefetch_tmap(lane == 0 ? &q_map : (lane == 1 ? &k_map : &v_map));
    if (warp == 9) tmem_alloc(&sm.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = sm.tmem;
    // ---- places of the entries on the line, and parts before each (a block-wide scan; every CTA stores the same)
    const int entries = a.num_groups + a.num_seqs;
    int64_t line = 0, len = 0, parts = 0;
    int e_mine = -1;
    SharedEntry y{};  // the thread's entry of the last round
    for (int base = 0; base < entries; base += kThreads) {
        const int e = base + tid;
        int items = 0;
        len = 0;
        e_mine = -1;
        if (e < entries) {
            bool bad;
            const DsEntry x = ds_entry(a, e, bad);
            const DsSize s = ds_size(a, x, NK);
            len = static_cast<int64_t>(a.H) * s.units * s.unit;
            items = a.H * s.units;
            e_mine = e;
            y = SharedEntry{0, 0, x.b, x.row, x.rows, x.key, x.end};
            if (blockIdx.x == 0) {
                if (e >= a.num_groups && x.rows > 0)  // the rows' own positions, which the join reads
                    bad |= block_row(a.cache, x.b, x.end & ~(kBlock - 1)) < 0 ||
                           block_row(a.cache, x.b, (x.end + x.rows - 1) & ~(kBlock - 1)) < 0;
                if (bad) atomicOr(&sm.err, kErrBadMetadata);
            }
        }
        int64_t incl = len;
        int incl_items = items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, static_cast<long long>(incl), o);
            const int w = __shfl_up_sync(0xffffffffu, incl_items, o);
            if (lane >= o) {
                incl += v;
                incl_items += w;
            }
        }
        if (lane == 31) {
            sm.scan_line[warp] = incl;
            sm.scan_items[warp] = incl_items;
        }
        __syncthreads();
        int64_t before = line, before_items = parts;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) {
                before += sm.scan_line[w];
                before_items += sm.scan_items[w];
            }
            line += sm.scan_line[w];
            parts += sm.scan_items[w];
        }
        y.line = before + incl - len;
        y.parts = static_cast<int32_t>(before_items + incl_items - items);
        if (e < entries) {
            a.entries[e] = y;
            if (e == a.num_groups) sm.group_parts = before_items + incl_items - items;
        }
        __syncthreads();
    }
    // More parts than the host's bounds allow for, as groups that overlap can make (their starts do not ascend): nothing is done.
    // (Sums over a warp's entries are below 2^31, over all of them maybe not.)
    const int64_t group_parts = sm.group_parts;  // (a problem has a sequence)
    const bool over = group_parts > a.group_parts_most || parts - group_parts > a.seq_parts_most;
    if (tid == 0) a.entries[entries] = SharedEntry{line, static_cast<int32_t>(parts), over ? -1 : 0, 0, 0, 0, 0};
    if (over) {
        if (tid == 0) atomicOr(&sm.err, kErrBadMetadata);
        line = 0;
    }
    const int shares = ds_shares(line, gridDim.x);
    const bool idle = line == 0 || static_cast<int>(blockIdx.x) >= shares;
    const int64_t from = ds_cut(line, blockIdx.x, shares);
    // the entry where the share begins
    if (!idle && e_mine >= 0 && y.line <= from && from < y.line + len) {
        sm.first = e_mine;
        sm.first_entry = y;
    }
    for (int e = tid; !idle && e < (entries - 1) / kThreads * kThreads; e += kThreads) {  // (earlier rounds')
        if (a.entries[e].line <= from && from < a.entries[e + 1].line) {
            sm.first = e;
            sm.first_entry = ds_load(a.entries + e);
        }
    }
    __syncthreads();
    const int P = 128 / a.G;

    auto next_item = [&](int k, DsItem& x) {  // item k of the CTA, false where it never came
        if (!wait(&sm.info_full[k % kDsInfo], (k / kDsInfo) & 1)) return false;
        x = sm.info[k % kDsInfo];
        return true;
    };
    auto passed = [&](int k) { mbar_arrive(&sm.info_empty[k % kDsInfo]); };
    // One M tile: stage s takes every second key tile, of item k from tile (s + k) % 2 on.
    auto first_of = [](const DsItem& x, int k, int s) { return x.pair ? 0 : (s + k) & 1; };
    auto count_of = [](const DsItem& x, int k, int s) { return x.pair ? x.tiles : (x.tiles + 1 - ((s + k) & 1)) / 2; };

    if (idle) {
        // nothing to do
    } else if (warp >= 8) {
        if constexpr (kInt8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == 8 || warp == 10) {
            // ---------------- copies: K and V tiles, dimensions 0-63 by warp 8 (and the queries), 64-127 by warp 10 (which
            // also finds the items)
            const int half = warp == 10;
            int slot = 0, sent[3] = {0, 0, 0}, q_used[2] = {0, 0};  // copies in all and by barrier row; items by query buffer
            bool alive = true;
            // The CTA's walk along the line, piece after piece (of one KV head h, unit u and piece ch of the entry's keys; `at`
            // lies `on` tiles behind its beginning; `more`: the item has parts of this CTA); the entry after the present one
            // is loaded ahead.
            int64_t at = from;
            const int64_t stop = ds_cut(line, blockIdx.x + 1, shares);
            int e = sm.first, h = 0, u = 0, ch = 0, on = 0, more = 0;
            SharedEntry x = sm.first_entry, ahead = x;
            DsSize sz = ds_size(a, DsEntry{x.b, x.row, x.rows, x.key, x.end}, NK);
            if (half) {
                ahead = ds_load(a.entries + e + 1);
                const int off = static_cast<int>(at - x.line), uh = off / sz.unit, o = off - uh * sz.unit;
                h = uh / sz.units;
                u = uh - h * sz.units;
                ch = min(o / (kRun * sz.w + kDsExtra), sz.chunks - 1);
                on = o - ch * (kRun * sz.w + kDsExtra);
            }
            auto find = [&]() {
                DsItem it{};
                it.b = -1;
                while (at < stop) {
                    while (sz.units == 0) {  // an entry without items (the line goes on: there is another)
                        x = ahead;
                        ++e;
                        ahead = ds_load(a.entries + min(e + 1, entries));
                        sz = ds_size(a, DsEntry{x.b, x.row, x.rows, x.key, x.end}, NK);
                    }
                    const int tiles = min(kRun, sz.tiles - ch * kRun), len = min(kDsExtra + tiles * sz.w - on, static_cast<int>(min(stop - at, INT64_C(1) << 30)));
                    const int t0 = ds_tiles_before(on - kDsExtra, sz.w), t1 = ds_tiles_before(on + len - kDsExtra, sz.w);
                    const bool some = t1 > t0;
                    if (some) {
                        const bool group = e < a.num_groups;
                        it.b = x.b;
                        it.row = x.row + u * 2 * P;
                        it.rows = x.rows - u * 2 * P;
                        it.h = h;
                        it.key = x.key + (ch * kRun + t0) * NK;
                        it.end = x.end;
                        it.tiles = t1 - t0;
                        it.pair = it.rows > P;
                        it.cap = group ? a.group_rows : a.seq_rows;
                        it.more = more;
                        more = 1;
                        const int64_t place = x.parts + (h * sz.units + u) + static_cast<int>(blockIdx.x);
                        it.part = group ? place * 2 * a.group_rows : a.seq_part0 + (place - group_parts) * 2 * a.seq_rows;
                    }
                    at += len;
                    on = 0;  // (the share ends here if the item does not)
                    if (++ch == sz.chunks) {
                        ch = more = 0;
                        if (++u == sz.units) {
                            u = 0;
                            if (++h == a.H) {
                                h = 0;
                                sz.units = 0;
                            }
                        }
                    }
                    if (some) break;
                }
                return it;
            };
            auto publish = [&](int n, const DsItem& item) {
                int ok = 1;
                if (lane == 0) {
                    if (n >= kDsInfo) ok = wait(&sm.info_empty[n % kDsInfo], ((n / kDsInfo) - 1) & 1);
                    if (ok) {
                        sm.info[n % kDsInfo] = item;
                        mbar_arrive(&sm.info_full[n % kDsInfo]);
                    }
                }
                return __shfl_sync(0xffffffffu, ok, 0) != 0;
            };
            DsItem item, after;
            if (half) {
                after = find();
                alive = publish(0, after);
            }
            for (int k = 0; alive; ++k) {
                if (half) {
                    item = after;
                    if (item.b < 0) break;
                } else {
                    alive = __all_sync(0xffffffffu, next_item(k, item));
                    if (!alive) break;
                    __syncwarp();
                    if (lane == 0) passed(k);
                    if (item.b < 0) break;
                    int ok = 1;
                    if (lane == 0) {
                        for (int s = 0; s < (item.pair ? 2 : 1); ++s) {
                            const int buf = item.pair ? s : k & 1, used = buf ? q_used[1] : q_used[0];
                            if (used > 0) ok = ok && wait(&sm.q_empty[buf], (used - 1) & 1);
                            if (!ok) break;
                            mbar_arrive_expect_tx(&sm.q_full[buf], 2 * P * a.G * 128);
                            for (int c = 0; c < 2; ++c)
                                tma_load_3d(sm.q[buf] + c * (kDsQBytes / 2), &q_map, &sm.q_full[buf], 64 * c, item.h * a.G, item.row + s * P);
                            if (buf) ++q_used[1];
                            else ++q_used[0];
                        }
                    }
                    alive = __shfl_sync(0xffffffffu, ok, 0) != 0;
                }
                constexpr int kBatch = 32 / (NK / kBlock);  // tiles whose cache rows the lanes hold
                int64_t row = 0;
                for (int j = 0; alive && j < item.tiles; ++j) {
                    if (j % kBatch == 0) {
                        const int t = item.key + j * NK + lane * kBlock;
                        row = a.cache_tokens;  // past the end: a box past the cache is zeros
                        if (lane < NK / kBlock * (item.tiles - j) && t < item.end) {
                            row = block_row(a.cache, item.b, t);
                            if (row < 0) {  // page outside the pool
                                atomicOr(&sm.err, kErrBadMetadata);
                                row = a.cache_tokens;
                            }
                        }
                    }
                    const int set = item.pair ? 0 : 1 + ((j + k) & 1);
#pragma unroll
                    for (int kind = 0; kind < 2; ++kind) {  // K, V
                        const int st = slot % kStages, copy = set == 0 ? sent[0] : (set == 1 ? sent[1] : sent[2]);
                        int64_t r[NK / kBlock];
#pragma unroll
                        for (int c = 0; c < NK / kBlock; ++c) r[c] = __shfl_sync(0xffffffffu, row, (j % kBatch) * (NK / kBlock) + c);
                        int ok = 1;
                        if (kInt8 && lane == 0) {  // a block of codes each, if the tile has two
                            const int at = slot % kCodes;
                            if (slot >= kCodes) ok = wait(&sm.code_empty[at], ((slot / kCodes) - 1) & 1);
                            if (ok && half >= NK / kBlock) {
                                mbar_arrive(&sm.code_full[at]);
                            } else if (ok) {
                                mbar_arrive_expect_tx(&sm.code_full[at], kBlock * kHeadDim);
                                tma_load_3d(sm.codes[at] + half * (kBlock * kHeadDim), kind == 0 ? &k_map : &v_map, &sm.code_full[at], 0, item.h,
                                            static_cast<int>(half < NK / kBlock ? r[half < NK / kBlock ? half : 0] : 0));
                            }
                        }
                        if (!kInt8 && lane == 0) {
                            uint64_t* bar = &sm.full[set][copy % kStages];
                            if (slot >= kStages) ok = wait(&sm.empty[st], ((slot / kStages) - 1) & 1);
                            if (ok) {
                                if (set > 0 && !half) mbar_arrive(&sm.empty[st]);  // (for the stage that does not take the tile)
                                mbar_arrive_expect_tx(bar, Cfg::kTile / 2);
#pragma unroll
                                for (int c = 0; c < NK / kBlock; ++c)
                                    tma_load_3d(sm.ring[st] + half * kHalf + c * (kBlock * 128), kind == 0 ? &k_map : &v_map, bar, 64 * half,
                                                item.h, static_cast<int>(r[c]));
                            }
                        }
                        ++slot;
                        if (set == 0) ++sent[0];
                        else if (set == 1) ++sent[1];
                        else ++sent[2];
                        if (!__shfl_sync(0xffffffffu, ok, 0)) {
                            alive = false;
                            break;
                        }
                    }
                    if (half && alive && j == min(1, item.tiles - 1)) {  // the next item, behind the first copies
                        after = find();
                        alive = publish(k + 1, after);
                    }
                }
            }
            if (lane == 0 && !half) {  // no copy in flight at the end
                for (int s = 0; s < 2; ++s) {
                    const int used = s ? q_used[1] : q_used[0];
                    if (used > 0) wait(&sm.q_full[s], (used - 1) & 1);
                }
                if constexpr (kInt8) {
                    for (int b = 0; b < kCodes && b < slot; ++b) wait(&sm.code_full[b], ((slot - 1 - b) / kCodes) & 1);
                } else {
#pragma unroll
                    for (int s = 0; s < 3; ++s)
                        for (int b = 0; b < kStages && b < sent[s]; ++b) wait(&sm.full[s][b], ((sent[s] - 1 - b) / kStages) & 1);
                }
            }
        } else if (kInt8 && warp >= 12) {
            // ---------------- codes to bf16, exactly: a thread a key (64-key tiles: half a key), which also puts its scales down
            const int t = tid - 384, key = t % NK, piece = t / NK;
            int slot = 0, tiles = 0, sent[3] = {0, 0, 0};
            bool alive = true;
            for (int k = 0; alive; ++k) {
                DsItem item;
                alive = __all_sync(0xffffffffu, next_item(k, item));
                if (!alive) break;
                __syncwarp();
                if (lane == 0) passed(k);
                if (item.b < 0) break;
                // Scales of the thread's key in tile j (zeros past the end: their weights are zero whatever lies there); the lanes
                // hold the cache rows of the next 32 blocks.
                constexpr int kBatch = 32 / (NK / kBlock);
                int64_t row = -1;
                auto rows_from = [&](int j) {
                    const int p = item.key + j * NK + lane * kBlock;
                    row = j < item.tiles && p < item.end ? block_row(a.cache, item.b, p) : -1;
                };
                auto scales_of = [&](int j) {
                    const int64_t r = __shfl_sync(0xffffffffu, row, (j % kBatch) * (NK / kBlock) + key / kBlock);
                    const int p = item.key + j * NK + key;
                    float2 y = make_float2(0.f, 0.f);
                    if (j < item.tiles && p < item.end && r >= 0) {
                        const int64_t at = (r + (key & (kBlock - 1))) * a.H + item.h;
                        y = make_float2(a.k_scale[at], a.v_scale[at]);
                    }
                    return y;
                };
                rows_from(0);
                float2 next = scales_of(0);
                for (int j = 0; alive && j < item.tiles; ++j, ++tiles) {
                    const int set = item.pair ? 0 : 1 + ((j + k) & 1);
                    if (piece == 0) {
                        sm.sc[tiles % Cfg::kScales][0][key] = next.x;
                        sm.sc[tiles % Cfg::kScales][1][key] = next.y;
                    }
                    if ((j + 1) % kBatch == 0) rows_from(j + 1);
                    next = scales_of(j + 1);
#pragma unroll 1
                    for (int kind = 0; kind < 2; ++kind, ++slot) {
                        const int st = slot % kStages, from = slot % kCodes, copy = set == 0 ? sent[0] : (set == 1 ? sent[1] : sent[2]);
                        const bool ok = wait(&sm.code_full[from], (slot / kCodes) & 1) && (slot < kStages || wait(&sm.empty[st], ((slot / kStages) - 1) & 1));
                        alive = __all_sync(0xffffffffu, ok);
                        if (!alive) break;
                        if (set > 0 && t == 0) mbar_arrive(&sm.empty[st]);  // (for the stage that does not take the tile)
                        // (64-key tiles: a half of the dimensions a thread)
                        const uint32_t x16 = (key & 7) << 4;
                        uint32_t src = smem_u32(sm.codes[from]) + key * kHeadDim, dst = smem_u32(sm.ring[st]) + key * 128 + piece * kHalf;
#pragma unroll 1
                        for (int c0 = piece * (NK / 16); c0 < (piece + 1) * (NK / 16); c0 += 4, dst += kHalf) {  // 64 dims
#pragma unroll
                            for (int i = 0; i < 4; i += 2) {
                                uint4 w[2];
#pragma unroll
                                for (int n = 0; n < 2; ++n) w[n] = ds_ld_shared(src + (((c0 + i + n) << 4) ^ x16));
#pragma unroll
                                for (int n = 0; n < 2; ++n) {
                                    const uint32_t ws[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
                                    uint32_t o[8];
#pragma unroll
                                    for (int x = 0; x < 4; ++x) {
                                        const uint32_t even = i8_even_to_bf16(ws[x]), odd = i8_even_to_bf16(ws[x] >> 8);
                                        o[2 * x] = __byte_perm(even, odd, 0x5410);
                                        o[2 * x + 1] = __byte_perm(even, odd, 0x7632);
                                    }
                                    ds_st_shared(dst + ((2 * (i + n)) << 4 ^ x16), make_uint4(o[0], o[1], o[2], o[3]));
                                    ds_st_shared(dst + ((2 * (i + n) + 1) << 4 ^ x16), make_uint4(o[4], o[5], o[6], o[7]));
                                }
                            }
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sm.full[set][copy % kStages]);
                            mbar_arrive(&sm.code_empty[from]);
                        }
                        if (set == 0) ++sent[0];
                        else if (set == 1) ++sent[1];
                        else ++sent[2];
                    }
                }
            }
        } else {
            // ---------------- matrix instructions of stage s, one thread
            const int s = warp == 9 ? 0 : 1;
            if (lane == 0) {
                constexpr uint32_t idesc_s = idesc_bf16_f32(128, NK, 0, 0), idesc_o = idesc_bf16_f32(128, kHeadDim, 0, 1);
                const uint64_t qd0 = smem_desc_sw128(smem_u32(sm.q[0]), 16, 1024), qd1 = smem_desc_sw128(smem_u32(sm.q[1]), 16, 1024);
                const uint64_t kd = smem_desc_sw128(smem_u32(sm.ring[0]), 16, 1024);
                const uint64_t vd = smem_desc_sw128(smem_u32(sm.ring[0]), kHalf, 1024);
                // running: ring slots, the stage's tiles, turns taken, copies seen of pairs and of alternate tiles, query buffers
                int slots = 0, tiles = 0, turns = 0, seen[2] = {0, 0}, q_used[2] = {0, 0};
                bool ok = true, issued = false;
                for (int k = 0; ok; ++k) {
                    DsItem item;
                    ok = next_item(k, item);
                    if (!ok) break;
                    passed(k);
                    if (item.b < 0) break;
                    const int count = count_of(item, k, s), step = item.pair ? 1 : 2, j0 = first_of(item, k, s);
                    const bool pair = item.pair;
                    const int row = pair ? 0 : 1 + s;
                    auto landed = [&]() {  // the stage's next copy
                        int& n = pair ? seen[0] : seen[1];
                        const bool r = wait(&sm.full[row][n % kStages], (n / kStages) & 1);
                        ++n;
                        return r;
                    };
                    auto at = [&](int j, int kind) { return (slots + 2 * j + kind) % kStages; };
                    const int b0 = pair ? 0 : k & 1, b1 = pair ? 1 : k & 1;  // query buffers of the item
                    const uint64_t qd = (pair ? s : k & 1) ? qd1 : qd0;
                    auto free_q = [&](bool products) {
                        for (int b = b0; b <= b1; ++b) {
                            if (products) tc_commit(&sm.q_empty[b]);
                            else mbar_arrive(&sm.q_empty[b]);
                        }
                    };
                    for (int b = b0; b <= b1 && ok; ++b) {
                        int& n = b ? q_used[1] : q_used[0];
                        ok = wait(&sm.q_full[b], n & 1);
                        ++n;
                    }
                    if (!ok) break;
                    // S_s = Q K^T from ring slot st; `pass`: the other stage's turn begins while the last of them run
                    auto scores = [&](int st, bool last, bool pass) {
                        const uint64_t kb = kd + static_cast<uint64_t>(st * (Cfg::kTile >> 4));
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            tc_mma_ss(tmem + s * 128 + kSAt, qd + static_cast<uint64_t>(((i >> 2) * (kDsQBytes / 2) + (i & 3) * 32) >> 4),
                                      kb + static_cast<uint64_t>(((i >> 2) * kHalf + (i & 3) * 32) >> 4), idesc_s, i > 0);
                            if (i == 5 && pass) mbar_arrive(&sm.turn[s ^ 1]);
                        }
                        tc_commit(&sm.s_full[s]);
                        if (last) free_q(true);  // the last products with this item's queries
                        tc_commit(&sm.empty[st]);
                    };
                    if (count > 0) {
                        ok = landed();
                        if (!ok) break;
                        issued = true;
                        tc_fence_after();
                        scores(at(j0, 0), count == 1, false);
                    } else {
                        free_q(false);
                    }
                    // The other stage is through with the item before the last one (no barrier is then two phases behind), and for
                    // turns with the last one (its turns have been taken).
                    if (k > 1) ok = wait(&sm.item_done[k & 1], ((k >> 1) - 1) & 1);
                    if (pair && k > 0) ok = ok && wait(&sm.item_done[(k - 1) & 1], ((k - 1) >> 1) & 1);
                    for (int c = 0; ok && c < count; ++c) {
                        // pairs take turns: values of tile c, scores of the next (whatever can be waited for is, first)
                        const int j = j0 + step * c;
                        const uint32_t phase = (tiles + c) & 1;
                        const bool next = c + 1 < count, pass = pair && (s == 0 || next);
                        ok = landed();
                        const int st_v = at(j, 1), st_k = at(j + step, 0);
                        if (pair && next) ok = ok && landed();
                        const uint64_t vb = vd + static_cast<uint64_t>(st_v * (Cfg::kTile >> 4));
                        ok = ok && wait(&sm.p_full[s][0], phase);
                        if (ok && pair && (s == 1 || c > 0)) ok = wait(&sm.turn[s], turns++ & 1);
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
                                              !((kParts > 1 ? c % 2 == 0 : c == 0) && part == 0 && i == 0));
                        }
                        if (!ok) break;
                        if (!pair && next) {  // the values' slot back before the next keys are waited for
                            tc_commit(&sm.empty[st_v]);
                            ok = landed();
                            if (!ok) break;
                            tc_fence_after();
                        }
                        if (next) {
                            scores(st_k, c + 2 == count, pass);
                        } else {
                            if (pass) mbar_arrive(&sm.turn[s ^ 1]);
                            tc_commit(&sm.o_full[s]);
                        }
                        if (pair || !next) tc_commit(&sm.empty[st_v]);
                    }
                    slots += 2 * item.tiles;
                    tiles += count;
                    if (ok) mbar_arrive(&sm.item_done[k & 1]);
                }
                if (issued) {  // every matrix instruction done before tensor memory is given back
                    tc_commit(&sm.drain[s]);
                    wait(&sm.drain[s], 0);
                }
            }
            __syncwarp();
        }
    } else {
        // 168 x 384 registers at launch: 200 x 256 + 104 x 128; int8 128 x 512: 184 x 256 + 72 x 256
        if constexpr (kInt8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---------------- softmax group s: thread = row of its M tile
        const int s = warp >> 2, m = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // (32 (warp % 4)) << 16
        const uint32_t s_addr = tmem + s * 128 + lanes, o_addr = tmem + 256 + s * 128 + lanes;
        int tiles = 0, done = 0, before = 0, single = 0;  // running: the stage's tiles, items it had tiles of; key tiles of earlier items; the stage's of one M tile
        bool alive = true;
        for (int k = 0; alive; ++k) {
            DsItem item;
            alive = __all_sync(0xffffffffu, next_item(k, item));
            if (!alive) break;
            __syncwarp();
            if (lane == 0) passed(k);
            if (item.b < 0) break;
            const int count = count_of(item, k, s), j0 = first_of(item, k, s), step = item.pair ? 1 : 2;
            const int rows = min(item.rows - (item.pair ? s * P : 0), P) * a.G;  // of the M tile
            const bool mine = m < rows, busy = (m & ~31) < rows;                 // busy: some row of the warp is
            float top = -INFINITY, sum = 0.f;         // maximum in use (log2 domain), sum of weights
            float acc[kParts > 1 ? kHeadDim : 1];     // fp32 outputs: O of the row
            if constexpr (kParts > 1) {
#pragma unroll
                for (int d = 0; d < kHeadDim; ++d) acc[d] = 0.f;
            }
            auto rescale = [&](float r) {  // O in tensor memory times r
#pragma unroll 1
                for (int q = 0; q < kHeadDim / 32; ++q) {
                    float y[32];
                    dp_ld32(o_addr + 32 * q, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int d = 0; d < 32; ++d) y[d] *= r;
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
                        for (int d = 0; d < 16; ++d) acc[16 * q + d] += __uint_as_float(y[d]);
                    }
                }
            };
            for (int c = 0; alive && c < count; ++c) {
                const int t0 = item.key + (j0 + step * c) * NK;
                alive = __all_sync(0xffffffffu, wait(&sm.s_full[s], (tiles + c) & 1));
                if (!alive) break;
                const bool edge = t0 + NK > item.end;
                const int seen = item.end - t0;  // keys of the tile
                if (!kInt8 && edge && item.end % kBlock != 0) {
                    // Values past the end, which may be anything, become zero up to the end of their block (past the cache a copy
                    // fills with zeros).  One M tile: groups end with a block.
                    const int copy = 2 * (single + c) + 1, slot = (2 * (before + j0 + step * c) + 1) % kStages;
                    alive = __all_sync(0xffffffffu, wait(&sm.full[1 + s][copy % kStages], (copy / kStages) & 1));
                    if (!alive) break;
                    for (int y = seen * 16 + m; y < (seen + kBlock - 1) / kBlock * kBlock * 16; y += 128) {
                        const int key = y >> 4, part = y & 15;  // (a whole row: no swizzle to undo)
                        *reinterpret_cast<uint4*>(sm.ring[slot] + (part >> 3) * kHalf + key * 128 + (part & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (!busy) {  // (the tile's other warps have rows)
                    if (lane == 0) {
                        mbar_arrive(&sm.p_full[s][0]);
                        if constexpr (NK == 128) mbar_arrive(&sm.p_full[s][1]);
                    }
                    continue;
                }
                tc_fence_after();
                if (kParts > 1 && c > 0 && c % 2 == 0) collect();
                // int8: scales of the tile's keys and values
                const uint32_t k_sc = smem_u32(sm.sc[kInt8 ? (before + j0 + step * c) % Cfg::kScales : 0][0]), v_sc = k_sc + NK * 4;
                auto raise = [&](float now) {  // the maximum in use is now's or within kDsSlack of it
                    if (c == 0) {
                        top = now;
                    } else if (__any_sync(0xffffffffu, now > top + kDsSlack)) {
                        // the warp's rows of O move to the new maximum (no product runs on it now: S of this tile was computed
                        // after the last one), and their sums
                        const float next = now > top + kDsSlack ? now : top;
                        const float r = top == -INFINITY ? (next == -INFINITY ? 1.f : 0.f) : dp_exp2(top - next);
                        if constexpr (kParts > 1) {
#pragma unroll
                            for (int d = 0; d < kHeadDim; ++d) acc[d] *= r;
                            if (c & 1) rescale(r);
                        } else {
                            rescale(r);
                        }
                        sum *= r;
                        top = next;
                    }
                };
                if constexpr (kParts > 1) {  // ---- 32 scores at a time, O in registers
                    float now = -INFINITY;
                    auto scores_of = [&](int q, float (&x)[32]) {
                        dp_ld32(s_addr + kSAt + 32 * q, x);
                        tmem_ld_wait();
                        if constexpr (kInt8) {
                            ds_times32(x, k_sc + 128 * q);
                        }
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = 32 * q + i < seen ? x[i] * a.scale_log2 : -INFINITY;
                        }
                    };
                    const float f = edge ? 1.f : a.scale_log2;  // what is left to multiply by
                    if (kInt8 || edge) {
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {
                            float x[32];
                            scores_of(q, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) now = fmaxf(now, x[i]);
                        }
                        now *= f;
                    } else {
                        tmem_ld_max64(s_addr + kSAt, now);
                        tmem_ld_wait();
                        now *= f;
                    }
                    raise(now);
                    const float base = top == -INFINITY ? 0.f : top;
                    const float2 ff = make_float2(f, f), nb = make_float2(-base, -base);
                    float2 add = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        float x[32];
                        scores_of(q, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), ff, nb);
                            x[2 * i] = dp_exp2(y.x);
                            x[2 * i + 1] = dp_exp2(y.y);
                            add = __fadd2_rn(add, make_float2(x[2 * i], x[2 * i + 1]));
                        }
                        if constexpr (kInt8) {
                            ds_times32(x, v_sc + 128 * q);
                        }
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            uint32_t pk[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                pk[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                                if (part + 1 < kParts) {
                                    x[2 * i] -= bf16_lo(pk[i]);
                                    x[2 * i + 1] -= bf16_hi(pk[i]);
                                }
                            }
                            dp_st16(s_addr + part * 32 + 16 * q, pk);
                        }
                    }
                    sum += add.x + add.y;
                    dp_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[s][0]);
                } else {
                    float f = a.scale_log2;
                    if (edge) {  // keys past the end: the tile's scores as they are to be go back to where they are read from
#pragma unroll 1
                        for (int q = 0; q < NK / 32; ++q) {
                            float x[32];
                            dp_ld32(s_addr + 32 * q, x);
                            tmem_ld_wait();
                            if constexpr (kInt8) ds_times32(x, k_sc + 128 * q);
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                x[i] = 32 * q + i < seen ? x[i] * f : -INFINITY;
                            }
                            dp_st32(s_addr + 32 * q, reinterpret_cast<const uint32_t*>(x));
                        }
                        dp_st_wait();
                        f = 1.f;
                    }
                    float x[NK], big[NK / 64];
#pragma unroll
                    for (int q = 0; q < NK / 64; ++q) dp_ld64_max(s_addr + 64 * q, x + 64 * q, big[q]);
                    tmem_ld_wait();
                    float now;
                    if (kInt8 && !edge) {
#pragma unroll
                        for (int q = 0; q < NK / 32; ++q) ds_times32(x + 32 * q, k_sc + 128 * q);
                        float y[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                        for (int i = 4; i < NK; i += 4)
#pragma unroll
                            for (int z = 0; z < 4; ++z) y[z] = fmaxf(y[z], x[i + z]);
                        now = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * f;
                    } else {
                        now = fmaxf(big[0], big[NK / 64 - 1]) * f;
                    }
                    raise(now);
                    const float base = top == -INFINITY ? 0.f : top;
                    const float2 ff = make_float2(f, f), nb = make_float2(-base, -base);
                    float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int h2 = 0; h2 < NK / 64; ++h2) {  // 64 keys at a time: the products with them start while the next are made
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float* z = x + 64 * h2 + 32 * q;
                            uint32_t pk[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 y = __ffma2_rn(make_float2(z[2 * i], z[2 * i + 1]), ff, nb);
                                z[2 * i] = dp_exp2(y.x);
                                z[2 * i + 1] = dp_exp2(y.y);
                                add[i & 1] = __fadd2_rn(add[i & 1], make_float2(z[2 * i], z[2 * i + 1]));
                            }
                            if constexpr (kInt8) {
                                ds_times32(z, v_sc + 256 * h2 + 128 * q);
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(z[2 * i], z[2 * i + 1]);
                            dp_st16(s_addr + 32 * h2 + 16 * q, pk);
                        }
                        dp_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.p_full[s][h2]);
                    }
                    sum += (add[0].x + add[0].y) + (add[1].x + add[1].y);
                }
            }
            if (alive && count > 0) alive = __all_sync(0xffffffffu, wait(&sm.o_full[s], done++ & 1));
            tiles += count;
            before += item.tiles;
            if (!item.pair) single += count;
            if (!alive) break;
            if (!busy) continue;
            // ---------------- the part: O, maximum, sum
            tc_fence_after();
            const int64_t row0 = item.part + s * item.cap;
            float4* dst = reinterpret_cast<float4*>(a.part_o) + row0 * (kHeadDim / 4) + m;
            float2* ml = reinterpret_cast<float2*>(a.part_ml + (row0 + m) * 2);
            if (count > 0) collect();
            if (item.more) {  // a later piece: from tensor memory, whatever the form
                if constexpr (kParts > 1) {
#pragma unroll
                    for (int q = 0; q < kHeadDim / 32; ++q) dp_st32(o_addr + 32 * q, reinterpret_cast<const uint32_t*>(acc + 32 * q));
                    dp_st_wait();
                }
                constexpr auto add = kParts > 1 || kInt8 ? ds_call_add_piece : ds_add_piece;
                add(o_addr, dst, item.cap, ml, mine, count > 0 ? top : -INFINITY, count > 0 ? sum : 0.f);
                tc_fence_before();
                continue;
            }
            if (count > 0) {
#pragma unroll(kParts > 1 ? 4 : 1)
                for (int q = 0; q < kHeadDim / 32; ++q) {
                    float y[32];
                    if constexpr (kParts > 1) {
#pragma unroll
                        for (int d = 0; d < 32; ++d) y[d] = acc[32 * q + d];
                    } else {
                        dp_ld32(o_addr + 32 * q, y);
                        tmem_ld_wait();
                    }
                    if (mine) {
#pragma unroll
                        for (int d = 0; d < 8; ++d)
                            dst[static_cast<int64_t>(8 * q + d) * item.cap] = make_float4(y[4 * d], y[4 * d + 1], y[4 * d + 2], y[4 * d + 3]);
                    }
                    __syncwarp();  // the next load is the whole warp's
                }
            }
            tc_fence_before();
            if (mine) *ml = make_float2(count > 0 ? top : -INFINITY, count > 0 ? sum : 0.f);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0) a.err_slots[blockIdx.x] = sm.err;
}

// Joins the parts of a row's pairs of KV head h with the row's own keys.  CTA (row, h, z): a quarter or half of the 128
// dimensions, a thread 4 of them of one query head.
struct DsRun {  // parts of a row's M tile that lie behind one another: `count` of `cap` rows, `step` rows apart (none: 0)
    int64_t row0;
    int count, step, cap, m;  // m: row of its first head in a part
};

template <bool kInt8, int kResident>
__global__ void __launch_bounds__(256, kResident) dense_shared_join(const SharedArgs a, int grid, int NK) {
    __shared__ float own[kMaxGroup][kDecodeMaxRows];  // scores of the row's own keys (log2 domain)
    __shared__ int64_t own_row[kDecodeMaxRows];
    __shared__ DsRun runs[2];  // of the group's keys, of the sequence's own
    __shared__ int row_keys;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, h = blockIdx.y, r = blockIdx.x;
    // Where everything lies is found out by one warp (by all of them: 1,360 instructions a warp, and 37 us for 32 at 256 rows
    // of 4 x 16 heads, by itself).
    int lo = 0, g = -1, own_keys = 0;
    DsEntry x{};
    if (warp == 0) {  // ---- the row's sequence: the last that begins at or before it, 32 candidates at a time
        int hi = a.num_seqs;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const uint32_t le = __ballot_sync(0xffffffffu, at < hi && a.cu_rows[at] <= r);
            const int last = le ? 31 - __clz(le) : 0;
            lo += last * step;
            hi = min(lo + step, hi);
        }
        bool bad;
        x = ds_seq(a, lo, g, bad);
        const int keys = x.rows > 0 && r >= x.row && r < x.row + x.rows ? r - x.row + 1 : 0;  // its own: x.end .. x.end + keys - 1
        int64_t row = 0;
        if (lane < keys) {
            const int t = x.end + lane;
            row = block_row(a.cache, x.b, t & ~(kBlock - 1));
            if (row >= 0) row = (row + (t & (kBlock - 1))) * a.H + h;
        }
        own_keys = __any_sync(0xffffffffu, row < 0) ? 0 : keys;
        if (lane < own_keys) own_row[lane] = row;
        if (lane == 0) row_keys = own_keys;
    }
    __syncthreads();
    own_keys = row_keys;
    bool there = own_keys > 0;
    // ---- the row's own keys, while the parts are still being made (what came before dense_shared_kernel is done: its CTAs
    // wait for that before they let this kernel begin)
    const int64_t q_row = (static_cast<int64_t>(r) * a.H + h) * a.G;
    for (int i = warp; i < a.G * own_keys; i += warps) {
        const int gh = i / own_keys, key = i - gh * own_keys;
        const uint2 qw = *reinterpret_cast<const uint2*>(a.q + (q_row + gh) * kHeadDim + 4 * lane);
        float k[4], f = a.scale_log2;
        if constexpr (kInt8) {
            const char4 w = *reinterpret_cast<const char4*>(static_cast<const int8_t*>(a.k) + own_row[key] * kHeadDim + 4 * lane);
            k[0] = w.x, k[1] = w.y, k[2] = w.z, k[3] = w.w;
            f *= a.k_scale[own_row[key]];
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.k) + own_row[key] * kHeadDim + 4 * lane);
            k[0] = bf16_lo(w.x), k[1] = bf16_hi(w.x), k[2] = bf16_lo(w.y), k[3] = bf16_hi(w.y);
        }
        float y = fmaf(bf16_lo(qw.x), k[0], fmaf(bf16_hi(qw.x), k[1], fmaf(bf16_lo(qw.y), k[2], bf16_hi(qw.y) * k[3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (lane == 0) own[gh][key] = y * f;
    }
    __syncthreads();
    const int d4s = kHeadDim / 4 / gridDim.z, gh = tid % a.G, d4 = tid / a.G + blockIdx.z * d4s;
    if (tid >= a.G * d4s) there = false;
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const int mine = there ? own_keys : 0;
    for (int i = 0; i < mine; ++i) top = fmaxf(top, own[gh][i]);
    for (int i = 0; i < mine; ++i) {
        const float y = own[gh][i], w = top == -INFINITY ? (y == y ? 0.f : y) : dp_exp2(y - top);
        float v[4];
        if constexpr (kInt8) {
            const char4 c = *reinterpret_cast<const char4*>(static_cast<const int8_t*>(a.v) + own_row[i] * kHeadDim + 4 * d4);
            const float f = a.v_scale[own_row[i]];
            v[0] = c.x * f, v[1] = c.y * f, v[2] = c.z * f, v[3] = c.w * f;
        } else {
            const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.v) + own_row[i] * kHeadDim + 4 * d4);
            v[0] = bf16_lo(c.x), v[1] = bf16_hi(c.x), v[2] = bf16_lo(c.y), v[3] = bf16_hi(c.y);
        }
        sum += w;
        o.x = fmaf(w, v[0], o.x);
        o.y = fmaf(w, v[1], o.y);
        o.z = fmaf(w, v[2], o.z);
        o.w = fmaf(w, v[3], o.w);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (r == 0 && h == 0 && blockIdx.z == 0 && warp == 0) {  // what the CTAs found wrong
        uint32_t e = 0;
        for (int c = lane; c < grid; c += 32) e |= a.err_slots[c];
        e = __reduce_or_sync(0xffffffffu, e);
        if (lane == 0) *a.err = e;
    }
    if (own_keys == 0) return;
    // ---- the parts, those of the group's keys and then those of the sequence's
    const int groups = a.num_groups, entries = groups + a.num_seqs;
    if (warp == 0) {
        const bool group = lane == 0;
        const SharedEntry total = ds_load(a.entries + entries), y = ds_load(a.entries + (group && g >= 0 ? g : groups + lo));
        const int group_parts = a.entries[groups].parts;
        if (lane < 2) {
            DsRun out{};
            if (total.b < 0) {
                out.count = -1;  // more than the host's bounds allow for
            } else if (!group || g >= 0) {
                const DsSize s = ds_size(a, DsEntry{y.b, y.row, y.rows, y.key, y.end}, NK);
                const int i = r - y.row;
                if (s.units > 0 && i >= 0 && i < y.rows) {  // (rows outside: cu_rows does not ascend)
                    const int P = 128 / a.G, shares = ds_shares(total.line, grid);
                    const int tile = i < P ? 0 : i / P, u = tile / 2, uh = h * s.units + u;
                    const bool pair = y.rows - u * 2 * P > P;
                    out.cap = group ? a.group_rows : a.seq_rows;
                    out.m = (i - tile * P) * a.G;
                    const int64_t begin = y.line + static_cast<int64_t>(uh) * s.unit;
                    // the CTAs of its first and last tiles
                    const int c0 = ds_owner(total.line, begin + kDsExtra, shares), c1 = ds_owner(total.line, begin + s.unit - s.w, shares);
                    const int64_t place = y.parts + uh + c0;
                    out.row0 = (group ? place * 2 * out.cap : a.seq_part0 + (place - group_parts) * 2 * out.cap) + (pair ? tile & 1 : 0) * out.cap;
                    out.count = (c1 - c0 + 1) * (pair ? 1 : 2);  // (one M tile: both stages' parts)
                    out.step = pair ? 2 * out.cap : out.cap;
                }
            }
            runs[lane] = out;
        }
    }
    __syncthreads();
    if (runs[0].count < 0) return;
    for (int k = 0; k < 2 && there; ++k) {
        const DsRun run = runs[k];
        const int m = run.m + gh;
        constexpr int kAtOnce = kResident > 1 ? 4 : 8;
        for (int i0 = 0; i0 < run.count; i0 += kAtOnce) {
            float4 v[kAtOnce];
            float2 ml[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int64_t at = run.row0 + static_cast<int64_t>(min(i0 + q, run.count - 1)) * run.step;
                ml[q] = *reinterpret_cast<const float2*>(a.part_ml + (at + m) * 2);
                v[q] = reinterpret_cast<const float4*>(a.part_o)[at * (kHeadDim / 4) + static_cast<int64_t>(d4) * run.cap + m];
            }
            float most = top;
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) most = fmaxf(most, ml[q].x);
            const float f = top == -INFINITY ? 0.f : dp_exp2(top - most);
            if (top != -INFINITY) {
                sum *= f;
                o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            }
            top = most;
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                // A part without a key, or with none above -inf, says nothing (nor is its O read), unless its sum is NaN.  Any
                // other counts, also with a weight that is 0 in fp32: an infinite value in it shows.
                if (i0 + q >= run.count || (ml[q].x == -INFINITY && ml[q].y == ml[q].y)) continue;
                const float w = ml[q].x == -INFINITY ? ml[q].y : dp_exp2(ml[q].x - top);
                sum = fmaf(w, ml[q].y, sum);
                o.x = fmaf(w, v[q].x, o.x);
                o.y = fmaf(w, v[q].y, o.y);
                o.z = fmaf(w, v[q].z, o.z);
                o.w = fmaf(w, v[q].w, o.w);
            }
        }
    }
    if (!there) return;
    const float inv = 1.f / sum;
    const int64_t at = (q_row + gh) * kHeadDim + 4 * d4;
    if (a.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

template <int kParts, bool kInt8>
static cudaError_t launch_shared(const SharedArgs& a, int grid, cudaStream_t stream) {
    const size_t smem = sizeof(DsSmem<kParts, kInt8>) + 1024;
    auto* kernel = dense_shared_kernel<kParts, kInt8>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(DsCfg<kParts, kInt8>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, *a.q_map, *a.k_map, *a.v_map, a)) != cudaSuccess) return e;
    // the dimensions over two CTAs, over four of few rows (one: 78 us for 75 where 73 rows of 8 x 5 heads are joined)
    const int64_t blocks = static_cast<int64_t>(a.total_rows) * a.H;
    const int z = blocks * 4 <= 2 * device_sm_count() ? 4 : 2;
    const int threads = (a.G * (kHeadDim / 4 / z) + 31) / 32 * 32;
    cfg.gridDim = dim3(static_cast<unsigned>(a.total_rows), static_cast<unsigned>(a.H), static_cast<unsigned>(z));
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    // four CTAs an SM where they are many (three or five: 3% to 8% more at 73 and 256 rows); few take more loads at once, and
    // shared memory that they do not use, so that an SM need not divide it anew behind the first kernel (fp32, 16 rows: 37.0 and
    // 36.2 us; 73 rows, which are many: 70.8 and 72.0)
    const bool many = blocks > device_sm_count();
    cfg.dynamicSmemBytes = many ? 0 : 40000;
    auto* join = a.kv_int8 ? (many ? dense_shared_join<true, 4> : dense_shared_join<true, 1>)
                           : (many ? dense_shared_join<false, 4> : dense_shared_join<false, 1>);
    return cudaLaunchKernelEx(&cfg, join, a, grid, DsCfg<kParts, kInt8>::NK);
}

SharedRoom dense_shared_room(int num_seqs, int num_groups, int H, int G, int total_rows, int max_rows_per_seq, int max_group_rows,
                             int max_shared_len) {
    SharedRoom r;
    const int64_t P = 128 / G, units = total_rows / (2 * P) + num_groups;
    r.grid = std::min(device_sm_count(), kDenseMaxShares);
    r.group_parts = max_shared_len < kBlock ? 0 : units * H;
    r.seq_parts = static_cast<int64_t>(num_seqs) * H;
    r.group_rows = static_cast<int>(std::min(P, static_cast<int64_t>(max_group_rows)) * G);
    r.seq_rows = std::min(max_rows_per_seq, kDecodeMaxRows) * G;
    r.seq_part0 = (r.group_parts > 0 ? (r.group_parts + kDenseMaxShares) * 2 * r.group_rows : 0);
    r.rows = r.seq_part0 + (r.seq_parts + kDenseMaxShares) * 2 * r.seq_rows;
    return r;
}

cudaError_t run_dense_shared(const SharedArgs& a, int grid, cudaStream_t stream) {
    if (a.kv_int8) return a.out_bf16 ? launch_shared<1, true>(a, grid, stream) : launch_shared<3, true>(a, grid, stream);
    return a.out_bf16 ? launch_shared<1, false>(a, grid, stream) : launch_shared<3, false>(a, grid, stream);
}

}  // namespace msa
