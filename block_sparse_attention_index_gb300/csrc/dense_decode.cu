// Decode family of the attention over every cached position: the combine of its parts, and the launches.
#include "dense_decode.cuh"

namespace msa {

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
        const int mine = tid < a.num_seqs ? dd_units<false>(a, tid, tiles, bad) : 0;
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
        s = dd_seq<false>(a, lo);
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
        s = dd_seq<false>(a, lo);
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
    cudaError_t e = launch_dense_decode_kernel<H, kInt8, kParts, false>(a, grid, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
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
