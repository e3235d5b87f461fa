// Attention over every cached position for decode rows and drafted windows (1 to 8 rows a sequence) of a batch in which
// groups of sequences share a prefix: the prefix is read once for all rows of the group.
//   out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m),  x_t = scale log2(e) q.k_t over t <= p
// A softmax over a set of keys splits into parts (O, m, l: unnormalised sum, maximum, sum of weights) over any division
// of the keys, joined by weights 2^(m_i - m).  Here a row's keys are divided into its group's shared positions [0, S),
// which are this file's, and its sequence's own [S, p], which the streaming kernel of decode rows takes (dense_decode.cuh:
// 16 rows are all that share those, and its warps take a tile of keys each, where a tile of 128 rows would leave seven
// eighths of the softmax threads without a row: 2 to 3 us a tile of 128 keys and CTA, against 0.6).  Every row of a group
// sees all shared positions: no edge, and no later token's value is ever multiplied with.
//
// dense_shared_kernel.  An item is an M tile of 128 rows (row = neighbouring query rows x G heads of a KV head) or two of
// them, and its keys in tiles of NK:
//   S[128, NK] = Q K^T     operands from shared memory (TMA, 128-byte swizzle), S in tensor memory
//   P = 2^(x - m)          a thread a row, written over S (m is raised only where it would grow by more than 8)
//   O[128, 128] += P V     P from tensor memory, V as it lies
// Two stages of 128 columns of S and of O: two M tiles that take turns on the tensor pipe, or one M tile whose stages
// take alternate key tiles.  One CTA per SM; all items' key tiles lie on a line, item after item, that is cut into even
// shares (going on to another item counts as some tiles); a CTA's shares of items leave their parts in the workspace.
//
// dense_shared_join.  A CTA takes a row and a KV head: the places of its parts follow from the two kernels' lines by
// arithmetic (slot = item + CTA, which is different for every pair of them that meets, as both ascend along the line).
// This kernel's parts lie [dim / 4][row][4], so that the rows of a tile are stored and loaded in whole lines.
//
// Numerics.  bf16 outputs: weights as one bf16 (2^-8 at most, at random), and at most 32,768 keys to a part, as the
// tensor cores cut what an addition loses instead of rounding it (2^-24 an addition of 16 keys).  fp32 outputs: weights
// as three bf16 parts, NK = 64, O taken from tensor memory every second tile and summed in registers.
#include <algorithm>

#include "common.cuh"
#include "dense_decode.cuh"
#include "groups.cuh"
#include "internal.h"
#include "tensor_rows.cuh"

namespace msa {

constexpr int kDsThreads = 384;  // softmax groups: warps 0-3, 4-7; 8 and 10 copies (10: items too), 9 and 11 matrix instructions
constexpr int kDsQBytes = 128 * kHeadDim * 2;
constexpr int kDsPartKeys = 32768;  // most keys of a part
// What lies on the line, in about 0.3 us: a key tile of two M tiles 1.5 us (the tensor pipe), of one 1.2 (its copies), and
// going on to another item 2.5.
constexpr int kDsPairTile = 5, kDsTile = 4, kDsExtra = 8;
constexpr int kDsBatch = 8;         // items published at a time, two batches deep
constexpr float kDsSlack = 8.f;     // log2 by which the running maximum may lag

// A CTA's share of an item.
struct DsItem {
    int b;             // sequence whose table is read; < 0: no more items
    int row, rows;     // first query row of the item, query rows of its group from there on
    int h, key, end;   // KV head; first key of the share; end of the group's keys
    int tiles, pair;   // key tiles; two M tiles, or one whose stages take alternate key tiles
    int64_t part;      // first row of its parts in the workspace

    __device__ __forceinline__ int count(int s) const { return pair ? tiles : (tiles + 1 - s) / 2; }  // key tiles of stage s
};

template <int kParts>
struct DsCfg {
    static constexpr int NK = kParts == 1 ? 128 : 64;
    static constexpr int kTile = NK * kHeadDim * 2;  // bytes of a K or V tile
    static constexpr int kStages = 5 * (128 / NK);
    static constexpr int kSAt = kParts == 1 ? 0 : 64;  // column of S in its 128 (as in the prompt kernel: P's parts from 0 on)
};

template <int kParts>
struct __align__(1024) DsSmem {
    using Cfg = DsCfg<kParts>;
    uint8_t q[2][kDsQBytes];
    uint8_t ring[Cfg::kStages][Cfg::kTile];
    // Copies landed: of pairs [0], of the stages on alternate tiles [1], [2], each counted by itself, so that an issuer sees
    // all phases of the barriers that it waits for.
    uint64_t full[3][Cfg::kStages], empty[Cfg::kStages];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2][2], o_full[2], turn[2], drain[2];  // P: by halves of the key tile
    uint64_t info_full[2], info_empty[2], pair_done;
    DsItem info[2][kDsBatch];
    int32_t next;  // the CTA's first item
    uint32_t tmem, err;
    int64_t scan_line[kDsThreads / 32];
    int32_t scan_items[kDsThreads / 32];
};
static_assert(sizeof(DsSmem<1>) + 1024 <= 227 * 1024, "shared-prefix attention exceeds 227 KB of shared memory");
static_assert(sizeof(DsSmem<3>) + 1024 <= 227 * 1024, "shared-prefix attention (fp32) exceeds 227 KB of shared memory");

// What the join has to know of a row.
struct DsRow {
    int seq, group;             // seq < 0: it is no row, or its sequence's metadata is bad; group < 0: none
    int row, rows;              // its sequence's first row, rows
    int group_row, group_rows;  // its group's
    int shared, blocks;         // shared positions; blocks of its own
};
static_assert(sizeof(DsRow) == kDsRowBytes, "records of the rows");

// How a group lies on the line: its keys in `chunks`, each of them for the `units` items (of up to two M tiles) of every KV
// head one after the other.  These read the same keys, or the same tokens, and neighbours on the line run at the same time on
// neighbouring CTAs, so that all but the first find them in L2: chunks are about as long as a CTA's share of the line (64
// rows at 32,768, 4 items a head: 276 MB were read from DRAM with the items' keys whole, 182 with chunks; 167 are needed).
struct DsSize {
    int tiles, chunks, units, heads, weight;  // key tiles; chunks; items a head; KV heads; a key tile's length on the line

    __device__ __forceinline__ int start(int ch) const { return tiles * ch / chunks; }  // (2^15 tiles and 160 chunks at most)
    __device__ __forceinline__ int length(int ch) const { return start(ch + 1) - start(ch); }
    __device__ __forceinline__ int parts() const { return chunks * heads * units; }
    __device__ __forceinline__ int64_t all() const { return static_cast<int64_t>(heads * units) * (tiles * weight + chunks * kDsExtra); }
    // Where chunk ch begins, and where the tiles of its item u of head h do, after the item's kDsExtra.
    __device__ __forceinline__ int64_t begin(int ch) const { return static_cast<int64_t>(heads * units) * (start(ch) * weight + ch * kDsExtra); }
    __device__ __forceinline__ int64_t place(int h, int ch, int u) const {
        return begin(ch) + static_cast<int64_t>(h * units + u) * (length(ch) * weight + kDsExtra) + kDsExtra;
    }
    __device__ __forceinline__ int part(int h, int ch, int u) const { return (ch * heads + h) * units + u; }
};
__device__ __forceinline__ DsSize ds_size(const SharedArgs& a, int rows, int keys, int NK, int share) {
    DsSize s{};
    if (rows <= 0 || keys <= 0) return s;
    const int run = kDsPartKeys / NK, P = 128 / a.G, mt = (rows + P - 1) / P;
    s.tiles = (keys + NK - 1) / NK;
    s.weight = mt > 1 ? kDsPairTile : kDsTile;
    s.units = (mt + 1) / 2;
    s.heads = a.H;
    s.chunks = max((s.tiles + run - 1) / run, (s.tiles * s.weight + share / 2) / share);
    return s;
}

// CTAs that share a line, and where share c begins (the largest c whose share begins at or before a place: ds_owner).
__host__ __device__ __forceinline__ int ds_shares(int64_t line, int grid) {
    const int64_t n = line / (kDsExtra + 2 * kDsTile);
    return static_cast<int>(n < 1 ? 1 : (n < grid ? n : grid));
}
__device__ __forceinline__ int64_t ds_cut(int64_t line, int c, int shares) {
    if (line < INT32_MAX / 256) return static_cast<uint32_t>(line) * static_cast<uint32_t>(c) / static_cast<uint32_t>(shares);
    return line * c / shares;
}
__device__ __forceinline__ int ds_owner(int64_t line, int64_t at, int shares) {
    const int64_t x = (at + 1) * shares - 1;
    if (line < INT32_MAX / 256) return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(line));
    return static_cast<int>(x / line);
}

// Leaves the records of sequence b's rows.
__device__ __noinline__ void ds_record(const SharedArgs& a, int b) {
    const int c0 = a.groups.cu_rows[b], c1 = a.groups.cu_rows[b + 1], L = a.cache_lens[b], n = c1 - c0;
    DsRow r{};
    r.seq = -1;
    // every row gets a record, whatever the row counts are: rows of no sequence from the first or the last
    if (b == 0)
        for (int i = 0; i < min(c0, a.groups.total_rows); ++i) a.rows[i] = r;
    if (b == a.groups.num_seqs - 1)
        for (int i = max(c1, 0); i < a.groups.total_rows; ++i) a.rows[i] = r;
    const int S = shared_of(a.groups, b, r.group);
    if (n >= 1 && n <= min(a.max_rows_per_seq, kDecodeMaxRows) && c0 >= 0 && c1 <= a.groups.total_rows && L <= a.max_cache_len && L - n >= S) {
        r.seq = b;
        r.row = c0;
        r.rows = n;
        r.shared = S;
        r.blocks = (L + kBlock - 1) / kBlock - S / kBlock;
        Group x;
        if (r.group >= 0 && group_at(a.groups, r.group, x)) {
            r.group_row = x.row;
            r.group_rows = x.rows;
        }
    }
    for (int i = max(c0, 0); i < min(c1, a.groups.total_rows); ++i) a.rows[i] = r;
}

template <int kParts>
__global__ void __launch_bounds__(kDsThreads, 1) dense_shared_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                    const __grid_constant__ CUtensorMap k_map,
                                                                    const __grid_constant__ CUtensorMap v_map,
                                                                    const SharedArgs a) {
    using Cfg = DsCfg<kParts>;
    using Smem = DsSmem<kParts>;
    constexpr int NK = Cfg::NK, kStages = Cfg::kStages, kHalf = Cfg::kTile / 2, kSAt = Cfg::kSAt;
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &sm.err); };
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            for (int k = 0; k < 3; ++k) mbar_init(&sm.full[k][s], 2);  // two warps copy a half each
            mbar_init(&sm.empty[s], 2);                                // both issuers (alternate tiles: one, and the copier for the other)
        }
        mbar_init(&sm.pair_done, 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.info_full[s], 1);
            mbar_init(&sm.info_empty[s], 11);  // a copier, two issuers, eight softmax warps
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
        sm.next = 0;
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
    // ---- places of the groups on the line, and parts before each (a block-wide scan; every CTA stores the same)
    const int num = a.groups.num, P = 128 / a.G;
    const bool few = num <= kDsThreads;  // a thread a group
    Group mine{};
    bool my_bad = false;
    if (few && tid < num) my_bad = !group_at(a.groups, tid, mine);
    auto group_of = [&](int g, bool& bad) {
        if (few) {
            bad = my_bad;
            return mine;
        }
        Group x;
        bad = !group_at(a.groups, g, x);
        return x;
    };
    int64_t line = 0;
    for (int g = tid; g < num; g += kDsThreads) {
        bool bad;
        const Group x = group_of(g, bad);
        const DsSize s = ds_size(a, x.rows, x.shared, NK, INT32_MAX);
        line += static_cast<int64_t>(a.H) * s.units * (s.tiles * s.weight + kDsExtra);
        if (bad && blockIdx.x == 0) atomicOr(&sm.err, kErrBadMetadata);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) line += __shfl_xor_sync(0xffffffffu, static_cast<long long>(line), o);
    if (lane == 0) sm.scan_line[warp] = line;
    if (tid < kDsBatch) sm.info[0][tid].b = -1;
    __syncthreads();
    line = 0;
    for (int w = 0; w < kDsThreads / 32; ++w) line += sm.scan_line[w];
    const int share = static_cast<int>(max(int64_t{kDsExtra + 2 * kDsTile}, min(line / gridDim.x, int64_t{INT32_MAX / 2})));  // about
    __syncthreads();
    line = 0;
    int parts = 0, my_items = 0, my_count = 0;
    int64_t my_line = 0;
    DsSize my_size{};
    for (int base = 0; base < num; base += kDsThreads) {
        const int g = base + tid;
        int64_t length = 0;
        int items = 0;
        if (g < num) {
            bool bad;
            const Group x = group_of(g, bad);
            my_size = ds_size(a, x.rows, x.shared, NK, share);
            if (my_size.units > 0) {
                length = my_size.all();
                items = my_size.parts();
            }
        }
        int64_t incl = length;
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
        int64_t before = line;
        int before_items = parts;
        for (int w = 0; w < kDsThreads / 32; ++w) {
            if (w < warp) {
                before += sm.scan_line[w];
                before_items += sm.scan_items[w];
            }
            line += sm.scan_line[w];
            parts += sm.scan_items[w];
        }
        if (g < num) {
            my_line = before + incl - length;
            my_items = before_items + incl_items - items;
            my_count = items;
            a.line[g] = my_line;
            a.items[g] = my_items;
        }
        __syncthreads();
    }
    if (tid == 0) {
        a.line[num] = line;
        a.line[num + 1] = share;
        a.items[num] = parts;
    }
    if (parts > a.parts_most) {  // more than the host's bounds allow for
        if (tid == 0) atomicOr(&sm.err, kErrBadMetadata);
        line = 0;
    }
    const int shares = ds_shares(line, gridDim.x);
    const bool idle = line == 0 || static_cast<int>(blockIdx.x) >= shares;
    // ---- the CTA's share of the line.  Its items are numbered as their parts are, from the one that holds its beginning on.
    const int64_t from = idle ? 0 : ds_cut(line, blockIdx.x, shares), stop = idle ? 0 : ds_cut(line, blockIdx.x + 1, shares);
    auto first_item = [&](const DsSize& sz, int items, int64_t at_line) {
        const int64_t o = from - at_line;
        int ch = min(static_cast<int>(o * sz.chunks / sz.all()), sz.chunks - 1);
        while (ch > 0 && sz.begin(ch) > o) --ch;
        while (ch + 1 < sz.chunks && sz.begin(ch + 1) <= o) ++ch;
        const int length = sz.length(ch) * sz.weight + kDsExtra, off = static_cast<int>(o - sz.begin(ch));
        const int hu = min(off / length, sz.heads * sz.units - 1);
        // (a tile is the CTA's in whose share it begins: the item's last may have)
        return items + sz.part(0, ch, hu) + (off - hu * length > length - sz.weight ? 1 : 0);
    };
    auto item_of = [&](int part, const Group& x, const DsSize& sz, int items, int64_t at_line) {
        DsItem it{};
        it.b = -1;
        const int at = part - items, ch_h = at / sz.units, u = at - ch_h * sz.units, ch = ch_h / sz.heads, h = ch_h - ch * sz.heads;
        const int64_t begin = at_line + sz.place(h, ch, u), last = min(stop, begin + sz.length(ch) * sz.weight);
        const int t0 = from > begin ? static_cast<int>(from - begin + sz.weight - 1) / sz.weight : 0;
        const int t1 = last > begin ? static_cast<int>(last - begin + sz.weight - 1) / sz.weight : 0;
        if (t1 <= t0) return it;
        it.b = x.first;
        it.row = x.row + u * 2 * P;
        it.rows = x.rows - u * 2 * P;
        it.h = h;
        it.key = (sz.start(ch) + t0) * NK;
        it.end = x.shared;
        it.tiles = t1 - t0;
        it.pair = it.rows > P;
        it.part = (static_cast<int64_t>(part) + blockIdx.x) * 2 * a.stage_rows;
        return it;
    };
    if (few && !idle) {  // the first items, by the threads that have their entries
        if (my_count > 0 && from >= my_line && from < my_line + my_size.all())
            sm.next = first_item(my_size, my_items, my_line);
        __syncthreads();
        const int next = sm.next;
        for (int part = max(my_items, next); part < min(my_items + my_count, next + kDsBatch); ++part)
            sm.info[0][part - next] = item_of(part, mine, my_size, my_items, my_line);
    }
    __syncthreads();

    auto next_item = [&](int k, DsItem& x) {  // item k of the CTA, false where it never came
        const int n = k / kDsBatch;
        if (k % kDsBatch == 0 && !wait(&sm.info_full[n & 1], (n >> 1) & 1)) return false;
        x = sm.info[n & 1][k % kDsBatch];
        return true;
    };
    auto passed = [&](int k, const DsItem& x) {  // (one thread of the role) the item has been read: the last of its batch
        if (k % kDsBatch == kDsBatch - 1 || x.b < 0) mbar_arrive(&sm.info_empty[(k / kDsBatch) & 1]);
    };

    // (the records: by the softmax groups, which wait for their first products anyway)
    if (warp < 8)
        for (int b = blockIdx.x + tid * gridDim.x; b < a.groups.num_seqs; b += 256 * gridDim.x) ds_record(a, b);
    if (idle) {
        // nothing to do
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8 || warp == 10) {
            // ---------------- copies: K and V tiles, dimensions 0-63 by warp 8 (and the queries), 64-127 by warp 10 (and items)
            const int half = warp == 10;
            int slot = 0, sent[3] = {0, 0, 0}, q_used[2] = {0, 0};  // copies in all and by barrier row; items by query buffer
            int next = sm.next;
            bool more = true;  // items beyond the published ones
            // the last of table[0 .. num] that is at most x, 32 candidates at a time (a whole warp)
            auto last_of = [&](auto* table, auto x) {
                int lo = 0, hi = num;
                while (hi - lo > 1) {
                    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
                    const uint32_t le = __ballot_sync(0xffffffffu, at < hi && table[at] <= x);
                    lo += (31 - __clz(le)) * step;
                    hi = min(lo + step, hi);
                }
                return lo;
            };
            if (half && !few) {
                const int lo = last_of(a.line, from);
                Group x;
                group_at(a.groups, lo, x);
                next = first_item(ds_size(a, x.rows, x.shared, NK, share), a.items[lo], a.line[lo]);
            }
            auto publish = [&](int n) {  // batch n: a lane an item
                int ok = 1;
                if (lane == 0 && n >= 2) ok = wait(&sm.info_empty[n & 1], ((n >> 1) - 1) & 1);
                if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
                DsItem it{};
                it.b = -1;
                if (n == 0 && few) {
                    if (lane < kDsBatch) it = sm.info[0][lane];
                } else {
                    const int part = next + lane;
                    // the num of the items: among the 32 from the first one's on, or found one by one
                    const int e0 = last_of(a.items, min(next, parts - 1));
                    const int begins = e0 + lane <= num ? a.items[e0 + lane] : INT32_MAX;
                    int lo = e0;
                    bool found = false;
                    for (int i = 0; i < kDsBatch; ++i) {
                        const int n_le = __popc(__ballot_sync(0xffffffffu, begins <= next + i));
                        if (lane == i) {
                            lo = e0 + n_le - 1;
                            found = n_le < 32;
                        }
                    }
                    if (lane < kDsBatch && part < parts) {
                        if (!found) {
                            lo = e0;
                            for (int hi = num; hi - lo > 1;) {
                                const int mid = (lo + hi) >> 1;
                                if (a.items[mid] <= part) lo = mid; else hi = mid;
                            }
                        }
                        Group x;
                        group_at(a.groups, lo, x);
                        it = item_of(part, x, ds_size(a, x.rows, x.shared, NK, share), a.items[lo], a.line[lo]);
                    }
                }
                more = __popc(__ballot_sync(0xffffffffu, it.b >= 0)) == kDsBatch;
                next += kDsBatch;
                if (lane < kDsBatch) sm.info[n & 1][lane] = it;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.info_full[n & 1]);
                return true;
            };
            constexpr int kBatch = 32 / (NK / kBlock);  // tiles whose cache rows the lanes hold
            // the cache row of the lane's block of tiles j0 .. of an item, loaded before they are needed
            auto rows_of = [&](const DsItem& x, int j0) {
                int64_t row = a.cache_tokens;  // past the end: a box past the cache is zeros
                const int t = x.key + j0 * NK + lane * kBlock;
                if (x.b >= 0 && lane < NK / kBlock * (x.tiles - j0) && t < x.end) {
                    row = block_row(a.cache, x.b, t);
                    if (row < 0) {  // page outside the pool
                        atomicOr(&sm.err, kErrBadMetadata);
                        row = a.cache_tokens;
                    }
                }
                return row;
            };
            bool alive = true;
            // the item at k, and the first cache rows of the one behind it (loaded an item ahead; none where the batch with it
            // is not there yet)
            auto item_at = [&](int k, DsItem& x) {
                if (half) {
                    x = sm.info[(k / kDsBatch) & 1][k % kDsBatch];
                    return true;
                }
                if (!__all_sync(0xffffffffu, next_item(k, x))) return false;
                __syncwarp();
                if (lane == 0) passed(k, x);
                return true;
            };
            DsItem item, after;
            if (half) alive = publish(0);
            if (alive) alive = item_at(0, item);
            int64_t row_next = alive ? rows_of(item, 0) : 0;
            for (int k = 0; alive && item.b >= 0; ++k) {
                int64_t row = row_next;
                // the next batch in the middle of this one: its place is free by then
                if (half && k % kDsBatch == kDsBatch / 2 && more && !publish(k / kDsBatch + 1)) break;
                if (!half) {
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
                    if (!alive) break;
                }
                alive = item_at(k + 1, after);
                if (!alive) break;
                row_next = item.tiles > kBatch ? rows_of(item, kBatch) : rows_of(after, 0);
                for (int j = 0; alive && j < item.tiles; ++j) {
                    if (j > 0 && j % kBatch == 0) {
                        row = row_next;
                        row_next = j + kBatch < item.tiles ? rows_of(item, j + kBatch) : rows_of(after, 0);
                    }
                    const int set = item.pair ? 0 : 1 + (j & 1);
#pragma unroll
                    for (int kind = 0; kind < 2; ++kind) {  // K, V
                        const int st = slot % kStages, copy = set == 0 ? sent[0] : (set == 1 ? sent[1] : sent[2]);
                        int64_t r[NK / kBlock];
#pragma unroll
                        for (int c = 0; c < NK / kBlock; ++c) r[c] = __shfl_sync(0xffffffffu, row, (j % kBatch) * (NK / kBlock) + c);
                        int ok = 1;
                        if (lane == 0) {
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
                }
                item = after;
            }
            if (lane == 0 && !half) {  // no copy in flight at the end
                for (int s = 0; s < 2; ++s) {
                    const int used = s ? q_used[1] : q_used[0];
                    if (used > 0) wait(&sm.q_full[s], (used - 1) & 1);
                }
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    for (int b = 0; b < kStages && b < sent[s]; ++b) wait(&sm.full[s][b], ((sent[s] - 1 - b) / kStages) & 1);
            }
        } else {
            // ---------------- matrix instructions of stage s, one thread
            const int s = warp == 9 ? 0 : 1;
            if (lane == 0) {
                constexpr uint32_t idesc_s = idesc_bf16_f32(128, NK, 0, 0), idesc_o = idesc_bf16_f32(128, kHeadDim, 0, 1);
                const uint64_t qd0 = smem_desc_sw128(smem_u32(sm.q[0]), 16, 1024), qd1 = smem_desc_sw128(smem_u32(sm.q[1]), 16, 1024);
                const uint64_t kd = smem_desc_sw128(smem_u32(sm.ring[0]), 16, 1024);
                const uint64_t vd = smem_desc_sw128(smem_u32(sm.ring[0]), kHalf, 1024);
                // running: ring slots, the stage's tiles, turns taken, pairs, copies seen of pairs and of alternate tiles, query buffers
                int slots = 0, tiles = 0, turns = 0, pairs = 0, seen[2] = {0, 0}, q_used[2] = {0, 0};
                bool ok = true, issued = false;
                for (int k = 0; ok; ++k) {
                    DsItem item;
                    ok = next_item(k, item);
                    if (!ok) break;
                    passed(k, item);
                    if (item.b < 0) break;
                    const bool pair = item.pair;
                    const int count = item.count(s), step = pair ? 1 : 2, j0 = pair ? 0 : s;
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
                    // the other stage is through with its last pair: its turns have been taken
                    if (pair && pairs > 0) ok = wait(&sm.pair_done, (pairs - 1) & 1);
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
                    if (pair) {
                        ++pairs;
                        if (ok) mbar_arrive(&sm.pair_done);
                    }
                }
                if (issued) {  // every matrix instruction done before tensor memory is given back
                    tc_commit(&sm.drain[s]);
                    wait(&sm.drain[s], 0);
                }
            }
            __syncwarp();
        }
    } else {
        // 168 x 384 registers at launch: 208 x 256 + 88 x 128
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---------------- softmax group s: thread = row of its M tile
        const int s = warp >> 2, m = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // (32 (warp % 4)) << 16
        const uint32_t s_addr = tmem + s * 128 + lanes, o_addr = tmem + 256 + s * 128 + lanes;
        int tiles = 0, done = 0;  // running: the stage's tiles, items it had tiles of
        bool alive = true;
        for (int k = 0; alive; ++k) {
            DsItem item;
            alive = __all_sync(0xffffffffu, next_item(k, item));
            if (!alive) break;
            __syncwarp();
            if (lane == 0) passed(k, item);
            if (item.b < 0) break;
            const bool pair = item.pair;
            const int count = item.count(s);
            const int rows = min(item.rows - (pair ? s * P : 0), P) * a.G;       // of the M tile
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
                const int t0 = item.key + (pair ? c : 2 * c + s) * NK;
                alive = __all_sync(0xffffffffu, wait(&sm.s_full[s], (tiles + c) & 1));
                if (!alive) break;
                if (!busy) {  // (the tile's other warps have rows)
                    if (lane == 0) {
                        mbar_arrive(&sm.p_full[s][0]);
                        if constexpr (NK == 128) mbar_arrive(&sm.p_full[s][1]);
                    }
                    continue;
                }
                tc_fence_after();
                if (kParts > 1 && c > 0 && c % 2 == 0) collect();
                const bool edge = t0 + NK > item.end;
                const int seen = item.end - t0;  // keys of the tile
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
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = 32 * q + i < seen ? x[i] * a.scale_log2 : -INFINITY;
                        }
                    };
                    const float f = edge ? 1.f : a.scale_log2;  // what is left to multiply by
                    if (edge) {
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {
                            float x[32];
                            scores_of(q, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) now = fmaxf(now, x[i]);
                        }
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
                    float x[NK], big[NK / 64];
#pragma unroll
                    for (int q = 0; q < NK / 64; ++q) dp_ld64_max(s_addr + 64 * q, x + 64 * q, big[q]);
                    float f = a.scale_log2;
                    tmem_ld_wait();
                    float now;
                    if (edge) {  // keys past the end; the scores are then not those that the load took the maximum of
#pragma unroll
                        for (int i = 0; i < NK; ++i) x[i] = i < seen ? x[i] * f : -INFINITY;
                        f = 1.f;
                        float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < NK; i += 4)
#pragma unroll
                            for (int z = 0; z < 4; ++z) y[z] = fmaxf(y[z], x[i + z]);
                        now = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
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
            if (!alive) break;
            if (!busy) continue;
            // ---------------- the part: O, maximum, sum
            tc_fence_after();
            const int64_t row0 = item.part + s * a.stage_rows;
            float4* dst = reinterpret_cast<float4*>(a.part_o) + row0 * (kHeadDim / 4) + m;
            if (count > 0) {
                collect();
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
                            dst[static_cast<int64_t>(8 * q + d) * a.stage_rows] = make_float4(y[4 * d], y[4 * d + 1], y[4 * d + 2], y[4 * d + 3]);
                    }
                    __syncwarp();  // the next load is the whole warp's
                }
            }
            tc_fence_before();
            if (mine) *reinterpret_cast<float2*>(a.part_ml + (row0 + m) * 2) = make_float2(count > 0 ? top : -INFINITY, count > 0 ? sum : 0.f);
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

// Joins the parts of a row's pairs of KV head h.  CTA (row, h, z): a share of the 128 dimensions, a thread 4 kD4 of them of
// one query head.  kDjList parts at a time: one warp finds where they are, the threads fetch their maxima and sums together,
// then every thread what has a weight, eight in flight.  What bounds it is that chain of loads.
constexpr int kDjThreads = 128;
constexpr int kDjList = 64;
struct DjPart {
    int64_t row, at;  // query head 0: its row for maximum and sum, its first four dimensions of O (in fours)
    int run;          // fours from one run of four dimensions to the next: the rows of a stage; own positions 1
    int first, end;   // query heads that it has
};
template <int kD4>
__global__ void __launch_bounds__(kDjThreads, 5) dense_shared_join(const __grid_constant__ SharedArgs a, int grid, int own_grid, int NK) {
    __shared__ DjPart part[kDjList];
    __shared__ float2 part_ml[kDjList][kMaxGroup];  // maximum and sum
    __shared__ int found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y, r = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t* segs = a.own_units + a.groups.num_seqs + 1;
    if (r == 0 && h == 0 && blockIdx.z == 0 && warp == 1) {  // what the CTAs found wrong
        uint32_t e = 0;
        for (int c = lane; c < grid; c += 32) e |= a.err_slots[c];
        for (int c = lane; c < own_grid; c += 32) e |= a.own_err_slots[c];
        e = __reduce_or_sync(0xffffffffu, e);
        if (lane == 0) *a.err = e;
    }
    const int64_t line = a.line[a.groups.num];
    const int share = static_cast<int>(a.line[a.groups.num + 1]), all_parts = a.items[a.groups.num];
    const int64_t own_units = a.own_units[a.groups.num_seqs], own_segs = segs[a.groups.num_seqs];
    const DsRow w = a.rows[r];
    // (sequences whose rows overlap may have written a record together: nothing is read outside the buffers all the same)
    if (w.seq < 0 || w.seq >= a.groups.num_seqs || w.group >= a.groups.num || w.rows > kDecodeMaxRows || r < w.row || r - w.row >= w.rows) return;
    if (all_parts > a.parts_most) return;
    constexpr int kD4s = kHeadDim / 4 / kD4;  // threads a query head, all CTAs of the row together
    const int per = kD4s / gridDim.z;
    const bool busy = tid < a.G * per;
    const int gh = busy ? tid % a.G : 0, d4 = (busy ? tid / a.G : 0) + blockIdx.z * per;  // the thread's: d4 + i kD4s
    const DsSize size = ds_size(a, w.group >= 0 ? w.group_rows : 0, w.shared, NK, share);
    const int chunks = size.units > 0 ? size.chunks : 0;
    float top = -INFINITY, sum = 0.f;
    float4 o[kD4];
#pragma unroll
    for (int d = 0; d < kD4; ++d) o[d] = make_float4(0.f, 0.f, 0.f, 0.f);
    // what is to be listed: a lane a chunk of the group's, then two tiles of 16 (row, head) pairs of its own positions
    for (int n0 = 0, n = kDjList; n == kDjList; n0 += kDjList) {  // parts n0 .. of the row's
        if (warp == 0) {
            int before = 0;
            for (int c0 = 0; c0 < chunks + 2 && before < n0 + kDjList; c0 += 32) {
                const int c = c0 + lane, i = r - w.row;
                int count = 0;
                int64_t step = 0;
                DjPart x{0, 0, 1, 0, a.G};
                if (c < chunks) {
                    const int at = r - w.group_row, P = 128 / a.G, tile = at / P, u = tile / 2, shares = ds_shares(line, grid);
                    const bool pair = w.group_rows - u * 2 * P > P;
                    const int64_t t0 = a.line[w.group] + size.place(h, c, u);
                    const int from = ds_owner(line, t0, shares), to = ds_owner(line, t0 + (size.length(c) - 1) * size.weight, shares);
                    const int64_t place = static_cast<int64_t>(a.items[w.group]) + size.part(h, c, u) + from;
                    const int64_t row0 = place * 2 * a.stage_rows + (pair ? (tile & 1) * a.stage_rows : 0);
                    count = (to - from + 1) * (pair ? 1 : 2);
                    step = pair ? 2 * a.stage_rows : a.stage_rows;
                    x.row = row0 + (at - tile * P) * a.G;
                    x.at = row0 * (kHeadDim / 4) + (at - tile * P) * a.G;
                    x.run = a.stage_rows;
                    if (at < 0 || at >= w.group_rows || row0 < 0 || row0 + static_cast<int64_t>(count) * step > a.part_rows) count = 0;
                } else if (c < chunks + 2) {
                    const int mt = i * a.G / 16 + c - chunks, tiles = (w.rows * a.G + 15) / 16, first = mt * 16 - i * a.G;
                    x.first = max(0, first);
                    x.end = min(a.G, first + 16);
                    if (mt < tiles && x.first < x.end && w.blocks > 0) {
                        const int extra = dd_extra(a.kv_int8);
                        const int64_t total = own_units * a.H, own_line = total + own_segs * extra;
                        const int shares = dd_shares(total, own_grid), n_seg = w.blocks * a.H, seg = segs[w.seq] + mt;
                        const int64_t at = static_cast<int64_t>(a.own_units[w.seq]) * a.H + static_cast<int64_t>(segs[w.seq]) * extra +
                                           static_cast<int64_t>(mt) * (n_seg + extra);
                        const int from = dd_div((at + 1) * shares - 1, own_line - extra), to = dd_div((at + n_seg) * shares - 1, own_line - extra);
                        const int64_t row0 = ((static_cast<int64_t>(seg) + from) * a.H + h) * 16;
                        count = to - from + 1;
                        step = 16 * a.H;
                        x.row = row0 - first;
                        x.at = x.row * (kHeadDim / 4);
                        if (row0 < 0 || row0 + (count - 1) * step + 16 > a.own_rows) count = 0;
                    }
                }
                int incl = count;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl += v;
                }
                const int first = before + incl - count;
                for (int q = max(0, n0 - first); q < min(count, n0 + kDjList - first); ++q) {
                    DjPart y = x;
                    y.row += q * step;
                    y.at += q * step * (kHeadDim / 4);
                    part[first + q - n0] = y;
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) found = min(kDjList, before - n0);
        }
        __syncthreads();
        n = found;
        for (int i = tid; i < n * a.G; i += kDjThreads) {
            const int q = i / a.G, gq = i - q * a.G;
            const DjPart x = part[q];
            const float* ml = x.run > 1 ? a.part_ml : a.own_ml;
            part_ml[q][gq] = gq >= x.first && gq < x.end ? *reinterpret_cast<const float2*>(ml + (x.row + gq) * 2) : make_float2(-INFINITY, 0.f);
        }
        __syncthreads();
        float most = top;
        for (int i = 0; i < n; ++i) most = fmaxf(most, part_ml[i][gh].x);
        if (most > top) {
            const float f = top == -INFINITY ? 0.f : dp_exp2(top - most);
            if (top != -INFINITY) {
                sum *= f;
#pragma unroll
                for (int d = 0; d < kD4; ++d) o[d] = make_float4(o[d].x * f, o[d].y * f, o[d].z * f, o[d].w * f);
            }
            top = most;
        }
        constexpr int kAtOnce = 8 / (kD4 > 2 ? 2 : 1);
        for (int i0 = 0; i0 < n; i0 += kAtOnce) {
            float4 v[kAtOnce][kD4];
            float f[kAtOnce], l[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int i = min(i0 + q, n - 1);
                const float2 ml = part_ml[i][gh];
                // a part with no key (maximum -inf) weighs nothing, unless its sum is NaN
                f[q] = i0 + q >= n ? 0.f : (ml.x == -INFINITY ? (ml.y == ml.y ? 0.f : ml.y) : dp_exp2(ml.x - top));
                l[q] = ml.y;
                const DjPart x = part[i];
#pragma unroll
                for (int d = 0; d < kD4; ++d) {
                    const int c = d4 + d * kD4s;
                    const float4* src = x.run > 1 ? reinterpret_cast<const float4*>(a.part_o) + x.at + gh + static_cast<int64_t>(c) * x.run
                                                  : reinterpret_cast<const float4*>(a.own_o) + x.at + gh * (kHeadDim / 4) + c;
                    if (f[q] != 0.f) v[q][d] = *src;
                }
            }
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                if (f[q] == 0.f) continue;
                sum = fmaf(f[q], l[q], sum);
#pragma unroll
                for (int d = 0; d < kD4; ++d) {
                    o[d].x = fmaf(f[q], v[q][d].x, o[d].x);
                    o[d].y = fmaf(f[q], v[q][d].y, o[d].y);
                    o[d].z = fmaf(f[q], v[q][d].z, o[d].z);
                    o[d].w = fmaf(f[q], v[q][d].w, o[d].w);
                }
            }
        }
        __syncthreads();  // before the list is made again
    }
    if (!busy) return;
    const float inv = 1.f / sum;
#pragma unroll
    for (int d = 0; d < kD4; ++d) {
        const int64_t at = ((static_cast<int64_t>(r) * a.H + h) * a.G + gh) * kHeadDim + 4 * (d4 + d * kD4s);
        if (a.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                make_uint2(pack_bf16x2(o[d].x * inv, o[d].y * inv), pack_bf16x2(o[d].z * inv, o[d].w * inv));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(o[d].x * inv, o[d].y * inv, o[d].z * inv, o[d].w * inv);
    }
}

template <int kParts>
static cudaError_t launch_shared(const SharedArgs& a, const DenseArgs& own, int grid, int own_grid, cudaStream_t stream) {
    const size_t smem = sizeof(DsSmem<kParts>) + 1024;
    auto* kernel = dense_shared_kernel<kParts>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kDsThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, *a.q_map, *a.k_map, *a.v_map, a)) != cudaSuccess) return e;
    if ((e = run_dense_decode_own(own, own_grid, stream)) != cudaSuccess) return e;
    // few rows: the dimensions over two or four CTAs a row and head, while all CTAs run at once (five an SM)
    const int64_t blocks = static_cast<int64_t>(a.groups.total_rows) * a.H, places = 5 * device_sm_count();
    const int z = blocks * 4 <= places ? 4 : (blocks * 2 <= places ? 2 : 1);
    cfg.gridDim = dim3(static_cast<unsigned>(a.groups.total_rows), static_cast<unsigned>(a.H), static_cast<unsigned>(z));
    cfg.blockDim = dim3(kDjThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    auto* join = z == 4 ? dense_shared_join<1> : z == 2 ? dense_shared_join<2> : dense_shared_join<4>;
    return cudaLaunchKernelEx(&cfg, join, a, grid, own_grid, DsCfg<kParts>::NK);
}

SharedRoom dense_shared_room(const GroupArgs& g, int H, int G, int max_rows_per_seq) {
    SharedRoom r;
    const int64_t P = 128 / G, units = g.total_rows / (2 * P) + g.num;
    // (chunks are at least half a share long where there are more of them than the longest parts make)
    r.parts = g.max_shared_len < kBlock ? 0 : units * H * ((g.max_shared_len + kDsPartKeys - 1) / kDsPartKeys) + 2 * kDenseMaxShares;
    r.stage_rows = std::max(2, static_cast<int>(std::min(P, static_cast<int64_t>(g.max_rows)) * G));  // (1 is the mark of own positions)
    r.rows = (r.parts + kDenseMaxShares) * 2 * r.stage_rows;
    const int64_t line = units * H * (((g.max_shared_len + 63) / 64) * kDsPairTile + kDsExtra);
    r.grid = ds_shares(line, std::min(device_sm_count(), kDenseMaxShares));
    const int64_t tiles = (static_cast<int64_t>(std::min(max_rows_per_seq, kDecodeMaxRows)) * G + 15) / 16;
    r.own_rows = (g.num_seqs * tiles + kDenseMaxShares) * H * 16;
    return r;
}

cudaError_t run_dense_shared(const SharedArgs& a, const DenseArgs& own, int grid, int own_grid, cudaStream_t stream) {
    return a.out_bf16 ? launch_shared<1>(a, own, grid, own_grid, stream) : launch_shared<3>(a, own, grid, own_grid, stream);
}

}  // namespace msa
