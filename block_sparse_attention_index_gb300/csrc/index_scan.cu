// Index scan of the decode family with the block max-pool fused in (as decode_scan.cu), for index keys of 8 bits, and for
// batches whose groups of sequences share a prefix:
//     m_j = max_{t in block j, t <= p}  iq[r,h,:] . ik[t,h,:],   ik = code 2^e (8 bits) or bf16
//
// Work unit = one 64-position block with all its index heads: of a group's shared positions, for all rows of the group, or
// of a sequence's own, for its 1 to 8 rows.  The units lie on a line, groups first, a unit for as long as it takes; one CTA
// per SM takes an even share and streams it through a ring of shared-memory stages (TMA boxes of 64 positions of a head,
// completing an mbarrier); a team of warps, one a head, owns every third stage (of four heads; a warp that takes a whole unit
// keeps its stage four times as long: 25 us for 19 where 32 rows share 65,536 positions).  Dot products run on mma.sync m16n8k16: A = 16 positions x 16 of the dimensions,
// held in registers for a whole head, B = eight query rows, taken one group of eight after the other.
//
// The order of the dimensions inside a dot product is free: lane `tig` of a row takes the 16 dimensions 16 tig .., which
// are one 16-byte load of codes, or two of bf16, and two of the queries.  Codes become bf16 exactly (7 instructions for 4);
// their power of two multiplies the finished scores, position by position, before the maximum: exact too, so that sums that
// are exact in 32 bits stay so (others differ in their last bits between kernels that add in another order).
//
// Bound by memory: 65 bytes a position and head with codes, 128 without; a group's are read once instead of once a
// sequence.  With many rows the products take over: eight rows of a head and a block are 16 mma and about 80 other
// instructions.
//
// Measured by itself, cold caches: 4 x 65,536 positions of 4 heads in codes, 22 us (68 MB; decode_scan's bf16 keys, twice the
// bytes, take 26), bound by its instructions (700 a head and block, 224 of them make bf16 of codes; 48 % issue); 32 rows that
// share 65,536 positions, bf16, 18 us.
#include "common.cuh"
#include "internal.h"

namespace msa {

template <int H, bool kShared, bool kInt8>
struct IxCfg {
    static constexpr int kKeyHeads = kShared ? 1 : H;
    static constexpr int kRowBytes = kInt8 ? kIndexDim : 2 * kIndexDim;
    static constexpr int kHeadBytes = kBlock * kRowBytes;  // [64 positions][64 dims]
    static constexpr int kUnitBytes = kKeyHeads * kHeadBytes;
    // Consumers: teams of a warp for each index head; a team takes every kTeams-th unit, in stages of its own.
    static constexpr int kTeam = kKeyHeads, kTeams = kKeyHeads >= 8 ? 1 : 12 / kKeyHeads, kConsumers = kTeam * kTeams;
    static constexpr int kStages = kUnitBytes >= 65536 ? 3 : (kUnitBytes >= 32768 ? (kInt8 ? 5 : 6) : (kUnitBytes >= 16384 && kInt8 ? 9 : 12));
    static_assert(kStages % kTeams == 0, "a stage belongs to one team");
    static constexpr int kThreads = 32 * (kConsumers + 1);  // and the producer
    // Codes of four heads and more: their exponents come into the stage too, a position's by a copy of 4 or 8 bytes (fewer
    // heads: by the consumers, a unit ahead).
    static constexpr bool kExpRing = kInt8 && kKeyHeads >= 4;
    static constexpr int kExpBytes = kExpRing ? kBlock * kKeyHeads : 0;
    static constexpr int kFullCount = kExpRing ? 33 : 1;
};

__device__ __forceinline__ uint4 ix_lds(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void ix_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr uint32_t kLineMost = 1u << 30;  // longer than any batch's line

// Entry e of the line: a group's shared positions or (behind the groups) a sequence's own.
struct IxEntry {
    int b;            // sequence whose table is read
    int row, rows;    // query rows
    int first, units; // blocks [first, first + units)
    int last;         // position of row 0 (groups: past all of them)
    int weight;       // of a unit on the line
};

// Group g; nothing of it is shared where its metadata is bad.
__device__ __forceinline__ IxEntry ix_group(const IndexScanArgs& a, int g, int& end, bool& bad) {
    IxEntry x{};
    const int b0 = a.group_starts[g], b1 = a.group_starts[g + 1], S = a.group_shared[g];
    end = 0;
    bad = b0 < 0 || b1 < b0 || b1 > a.num_seqs || S < 0 || S > a.max_shared_len;
    if (bad) return x;
    const int c0 = a.cu_rows[b0], c1 = a.cu_rows[b1];
    bad = c0 < 0 || c1 < c0 || c1 > a.total_rows || c1 - c0 > a.max_group_rows;
    if (bad) return x;
    end = b1;
    x.b = b0;
    x.row = c0;
    x.rows = c1 - c0;
    x.units = x.rows > 0 ? S / kBlock : 0;
    x.last = 1 << 30;
    x.weight = 2 + x.rows / 16;  // (halves of a sequence's unit; half as much a row or twice: 4% and 8% slower at 32 rows)
    return x;
}

// Sequence b: no units where it has no rows of this family or its metadata is bad (the attention that follows reports it).
__device__ __forceinline__ IxEntry ix_seq(const IndexScanArgs& a, int b) {
    IxEntry x{};
    const int r = a.cu_rows[b], n = a.cu_rows[b + 1] - r, L = a.cache_lens[b];
    int shared = 0;
    if (a.num_groups > 0) {
        int lo = 0, hi = a.num_groups, end;  // the last group that begins at or before b
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.group_starts[mid] <= b) lo = mid; else hi = mid;
        }
        bool bad;
        const IxEntry g = ix_group(a, lo, end, bad);
        if (b >= g.b && b < end) shared = g.units;
    }
    x.weight = 2;
    if (n < 1 || n > kDecodeMaxRows || n > a.rows_per_seq || r < 0 || r + n > a.total_rows || L < n || L > a.max_cache_len ||
        L - n < shared * kBlock || !seq_rows_ok(a.cache, b, L, a.cache_tokens))
        return x;
    x.b = b;
    x.row = r;
    x.rows = n;
    x.first = shared;
    x.units = (L + kBlock - 1) / kBlock - shared;
    x.last = L - n;
    return x;
}
__device__ __forceinline__ IxEntry ix_entry(const IndexScanArgs& a, int e) {
    if (e >= a.num_groups) return ix_seq(a, e - a.num_groups);
    int end;
    bool bad;
    return ix_group(a, e, end, bad);
}

// A warp's place among the CTA's units.
struct IxPlace {
    int e = -1, k = 0;  // entry, unit of it
    int at = 0;         // place on the line
    IxEntry x{};
};

template <int H, bool kShared, bool kInt8>
__global__ void __launch_bounds__(IxCfg<H, kShared, kInt8>::kThreads, 1) index_scan_kernel(const __grid_constant__ CUtensorMap ik_map,
                                                                                         const IndexScanArgs a) {
    using Cfg = IxCfg<H, kShared, kInt8>;
    constexpr int kStages = Cfg::kStages, kWarps = Cfg::kThreads / 32, KH = Cfg::kKeyHeads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* exps = ring + kStages * Cfg::kUnitBytes;  // [stage][position][head]
    uint64_t* full = reinterpret_cast<uint64_t*>(exps + kStages * Cfg::kExpBytes);
    uint64_t* empty = full + kStages;
    int32_t* line = reinterpret_cast<int32_t*>(empty + kStages);  // [entries + 1] places of the entries
    __shared__ int warp_tot[kWarps];
    __shared__ uint32_t err;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, entries = a.num_groups + a.num_seqs;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], Cfg::kFullCount);
            mbar_init(&empty[s], Cfg::kTeam);
        }
        fence_mbar_init();
        prefetch_tmap(&ik_map);
        err = 0;
    }
    __syncthreads();
    // (a programmatic dependent of what precedes it: inputs are read, and anything is written, from here on)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0)  // words that the kernels behind this one count in
        for (int i = tid; i < a.n_clear; i += Cfg::kThreads) a.clear_words[i] = 0;
    // exclusive sums over `count` values, in order, kThreads at a time; returns the sum
    auto scan = [&](int count, auto value, int32_t* to) {
        uint32_t carry = 0;
        for (int base = 0; base < count; base += Cfg::kThreads) {
            const int i = base + tid, mine = i < count ? value(i) : 0;
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) warp_tot[warp] = incl;
            __syncthreads();
            uint32_t before = carry;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += warp_tot[w];
                carry = min(carry + warp_tot[w], kLineMost);
            }
            if (i < count) to[i] = static_cast<int32_t>(before + incl - mine);
            __syncthreads();
        }
        return carry;
    };
    // The line of a batch within the host's bounds is shorter than 2^30 (4,096 sequences of 2^15 blocks, 2^15 rows of groups).
    // Groups that overlap, as their starts or cu_rows do not ascend, may make it longer (of 32 neighbours every second at
    // most is such a group: a warp's sum is below 2^31): nothing is scanned then.
    const uint32_t length = scan(entries, [&](int e) {
        const IxEntry x = ix_entry(a, e);
        return x.units * x.weight;
    }, line);
    const int total = length >= kLineMost ? 0 : static_cast<int>(length);
    if (tid == 0) {
        line[entries] = total;
        if (length >= kLineMost) atomicOr(&err, kErrBadMetadata);
    }
    if (blockIdx.x == 0) {
        if (a.drow_prefix != nullptr) {  // rows of the decode family before each sequence, for the attention's grid
            const uint32_t rows = scan(a.num_seqs, [&](int b) {
                const int n = a.cu_rows[b + 1] - a.cu_rows[b];
                return n >= 1 && n <= kDecodeMaxRows ? n : 0;
            }, a.drow_prefix);
            if (tid == 0) a.drow_prefix[a.num_seqs] = static_cast<int32_t>(rows);
        }
        for (int g = tid; g < a.num_groups; g += Cfg::kThreads) {
            int end;
            bool bad;
            ix_group(a, g, end, bad);
            if (bad) atomicOr(&err, kErrBadMetadata);
        }
        for (int b = tid; b < a.num_seqs && a.num_groups > 0; b += Cfg::kThreads)  // more rows than the bound, rows before the end of what is shared
            if (a.cu_rows[b + 1] != a.cu_rows[b] && ix_seq(a, b).rows == 0) atomicOr(&err, kErrBadMetadata);
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int from = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
    const int to = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
    // the first unit that begins in the share, and `steps` units on
    IxPlace place;
    auto enter = [&](int e) {
        place.e = e;
        place.x = ix_entry(a, e);
    };
    auto advance = [&](int steps) {
        place.k += steps;
        while (place.k >= place.x.units) {
            if (place.e + 1 >= entries) {
                place.at = INT32_MAX;
                return;
            }
            place.k -= place.x.units;
            enter(place.e + 1);
        }
        place.at = line[place.e] + place.k * place.x.weight;
    };
    if (from < to) {
        int lo = 0, hi = entries;  // the last entry that begins at or before the share
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (line[mid] <= from) lo = mid; else hi = mid;
        }
        enter(lo);
        advance((from - line[lo] + place.x.weight - 1) / place.x.weight);
    } else {
        place.at = INT32_MAX;
    }

    if (warp == Cfg::kConsumers) {
        // ---------------- producer: one lane streams units into the ring, all of them their exponents
        int i = 0;
        for (; place.at < to; ++i, advance(1)) {
            const int s = i % kStages;
            if (i >= kStages && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((i / kStages) - 1) & 1, &err))) break;
            int64_t row = block_row(a.cache, place.x.b, static_cast<int64_t>(place.x.first + place.k) * kBlock);
            if (row < 0) {  // page outside the pool
                if (lane == 0) atomicOr(&err, kErrBadMetadata);
                row = 0;
            }
            if constexpr (Cfg::kExpRing) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {  // (past the cache: zeros, and nothing is read)
                    const int64_t t = row + lane + 32 * y;
                    const uint32_t bytes = t < a.cache_tokens ? KH : 0;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(exps + s * Cfg::kExpBytes + (lane + 32 * y) * KH)),
                                 "l"(a.ik_exp + (bytes ? t : 0) * KH), "n"(KH >= 4 ? KH : 4), "r"(bytes)
                                 : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[s])) : "memory");
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], Cfg::kUnitBytes);
                // whole boxes: what lies past the sequence is masked, past the cache zeros
#pragma unroll
                for (int h = 0; h < KH; ++h)
                    tma_load_3d(ring + s * Cfg::kUnitBytes + h * Cfg::kHeadBytes, &ik_map, &full[s], 0, h, static_cast<int>(row));
            }
            __syncwarp();
        }
        // no copy in flight when the CTA ends
        for (int s = 0; s < kStages && s < i; ++s) mbar_wait(&full[s], ((i - 1 - s) / kStages) & 1, &err);
    } else {
        // ---------------- consumers.  Lane (grp, tig) = (lane / 4, lane % 4): of the products' B, column grp; of the
        // accumulators, positions 16 mt + grp and + 8, columns 2 tig and 2 tig + 1.
        constexpr int kTeams = Cfg::kTeams;
        const int grp = lane >> 2, tig = lane & 3, team = warp / Cfg::kTeam, h = warp % Cfg::kTeam;
        // codes: the head's exponents of positions lane and lane + 32, where they are loaded a unit ahead
        uint32_t ex[2] = {0, 0};
        auto load_exps = [&]() {
            if constexpr (kInt8 && !Cfg::kExpRing) {
                if (place.at >= to) return;
                const int64_t row = block_row(a.cache, place.x.b, static_cast<int64_t>(place.x.first + place.k) * kBlock);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int64_t t = max(row, int64_t{0}) + lane + 32 * y;
                    ex[y] = t < a.cache_tokens ? static_cast<uint8_t>(a.ik_exp[t * KH + h]) : 0;
                }
            }
        };
        // the queries of columns c0 .. c0 + 7, column grp's 16 dimensions of the lane
        auto load_queries = [&](const IxEntry& x, int columns, int c0, uint32_t (&qb)[8]) {
            const int col = min(c0 + grp, columns - 1);
            const uint4* src = reinterpret_cast<const uint4*>(
                a.iq + (static_cast<int64_t>(x.row) * H + (kShared ? col : static_cast<int64_t>(col) * H + h)) * kIndexDim + 16 * tig);
            const uint4 q0 = src[0], q1 = src[1];
            const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {  // codes: in their order
                qb[2 * kk] = kInt8 ? __byte_perm(w[2 * kk], w[2 * kk + 1], 0x5410) : w[2 * kk];
                qb[2 * kk + 1] = kInt8 ? __byte_perm(w[2 * kk], w[2 * kk + 1], 0x7632) : w[2 * kk + 1];
            }
        };
        uint32_t first_q[8];  // those of the entry's first eight columns
        int first_of = -1;
        if (place.at < to) advance(team);
        load_exps();
        for (int i = team; place.at < to; i += kTeams) {
            const IxEntry x = place.x;
            const int j = x.first + place.k, e_now = place.e, s = i % kStages;
            const uint32_t stage = smem_u32(ring + s * Cfg::kUnitBytes + h * Cfg::kHeadBytes);
            uint32_t now[2] = {ex[0], ex[1]};
            // columns: kShared one head's, (row, query head) pairs; else the rows of query head h
            const int columns = kShared ? x.rows * H : x.rows;
            if (e_now != first_of) {
                load_queries(x, columns, 0, first_q);
                first_of = e_now;
            }
            advance(kTeams);
            load_exps();
            if (!mbar_wait(&full[s], (i / kStages) & 1, &err)) break;
            if constexpr (Cfg::kExpRing) {
#pragma unroll
                for (int y = 0; y < 2; ++y) now[y] = exps[s * Cfg::kExpBytes + (lane + 32 * y) * KH + h];
            }
            const bool whole = x.last + 1 - j * kBlock >= kBlock;
            const int64_t slot = a.by_row ? x.row : static_cast<int64_t>(x.b) * a.rows_per_seq;  // of row 0 among the pooled scores
            uint32_t ka[4][4][4];  // A: [16 positions][16 of the lanes' dims]
            float power[4][2];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = mt * 16 + grp + 8 * e;
                    const uint32_t at = stage + row * Cfg::kRowBytes;
                    if constexpr (kInt8) {
                        const uint4 w = ix_lds(at + ((tig ^ ((row >> 1) & 3)) << 4));  // (64-byte swizzle)
                        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {  // dims 0 and 2, 1 and 3 of the four
                            ka[mt][kk][e] = i8_even_to_bf16(ws[kk]);
                            ka[mt][kk][2 + e] = i8_even_to_bf16(ws[kk] >> 8);
                        }
                    } else {
                        const uint4 w0 = ix_lds(at + (((2 * tig) ^ (row & 7)) << 4)), w1 = ix_lds(at + (((2 * tig + 1) ^ (row & 7)) << 4));
                        ka[mt][0][e] = w0.x, ka[mt][0][2 + e] = w0.y;
                        ka[mt][1][e] = w0.z, ka[mt][1][2 + e] = w0.w;
                        ka[mt][2][e] = w1.x, ka[mt][2][2 + e] = w1.y;
                        ka[mt][3][e] = w1.z, ka[mt][3][2 + e] = w1.w;
                    }
                }
            }
            if constexpr (kInt8) {
                // the lane's two positions' powers, then those of the accumulators' positions from their lanes
                float mine[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) mine[y] = index_power(static_cast<int8_t>(now[y]));
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) power[mt][e] = __shfl_sync(0xffffffffu, mine[mt >> 1], (mt & 1) * 16 + grp + 8 * e);
            }
            for (int c0 = 0; c0 < columns; c0 += 8) {
                uint32_t qb[8];
                if (c0 == 0) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) qb[kk] = first_q[kk];
                } else {
                    load_queries(x, columns, c0, qb);
                }
                float c[4][4];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) c[mt][0] = c[mt][1] = c[mt][2] = c[mt][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) ix_mma(c[mt], ka[mt][kk], qb[2 * kk], qb[2 * kk + 1]);
                // the lane's columns: rows' visible positions of the block (all of them in most blocks; the odd columns only where
                // there is more than one)
                float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (e == 1 && columns - c0 < 2) break;
                    if constexpr (kInt8) {
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt) {
                            c[mt][e] *= power[mt][0];
                            c[mt][2 + e] *= power[mt][1];
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt) m[e] = fmaxf(m[e], fmaxf(c[mt][e], c[mt][2 + e]));
                    } else {
                        const int ce = c0 + 2 * tig + e, seen = x.last + (kShared ? ce / H : ce) + 1 - j * kBlock;
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt) {
                            const int t = mt * 16 + grp;
                            if (t < seen) m[e] = fmaxf(m[e], c[mt][e]);
                            if (t + 8 < seen) m[e] = fmaxf(m[e], c[mt][2 + e]);
                        }
                    }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], o));
                }
                if (grp < 2) {  // lanes 0-3 store the even columns, 4-7 the odd ones
                    const int ce = c0 + 2 * tig + grp, i_row = kShared ? ce / H : ce;
                    if (ce < columns && x.last + i_row + 1 > j * kBlock)
                        a.pooled[(kShared ? slot * H + ce : (slot + ce) * H + h) * a.max_blocks + j] = grp ? m[1] : m[0];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);  // stage reusable
        }
    }
    __syncthreads();
    if (tid == 0) a.found[blockIdx.x] = err;  // what was found wrong
}

template <int H, bool kShared, bool kInt8>
static cudaError_t launch_index_scan(const IndexScanArgs& a, cudaStream_t stream) {
    using Cfg = IxCfg<H, kShared, kInt8>;
    const size_t smem = 1024 + static_cast<size_t>(Cfg::kStages) * (Cfg::kUnitBytes + Cfg::kExpBytes) + 2 * Cfg::kStages * sizeof(uint64_t) +
                        static_cast<size_t>(a.num_groups + a.num_seqs + 1) * sizeof(int32_t);
    auto* kernel = index_scan_kernel<H, kShared, kInt8>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(scan_grid(a.unit_bound)), 1, 1);
    cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, *a.ik_map, a);
}

template <int H>
static cudaError_t launch_index_scan_h(const IndexScanArgs& a, cudaStream_t stream) {
    if constexpr (H > 1) {
        if (a.ik_shared) return a.ik_exp ? launch_index_scan<H, true, true>(a, stream) : launch_index_scan<H, true, false>(a, stream);
    }
    return a.ik_exp ? launch_index_scan<H, false, true>(a, stream) : launch_index_scan<H, false, false>(a, stream);
}

cudaError_t run_index_scan(const IndexScanArgs& a, cudaStream_t stream) {
    switch (a.H) {
        case 1: return launch_index_scan_h<1>(a, stream);
        case 2: return launch_index_scan_h<2>(a, stream);
        case 4: return launch_index_scan_h<4>(a, stream);
        case 8: return launch_index_scan_h<8>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace msa
