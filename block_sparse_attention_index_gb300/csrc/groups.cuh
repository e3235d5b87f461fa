// Groups of sequences that share a prefix, as the kernels read them.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace msa {

struct Group {
    int first, last;  // sequences [first, last)
    int row, rows;    // query rows
    int shared;       // shared positions, in whole blocks
};

// Group g; false where its metadata is bad: then nothing of it is shared.
__device__ __forceinline__ bool group_at(const GroupArgs& a, int g, Group& x) {
    const int b0 = a.starts[g], b1 = a.starts[g + 1], S = a.shared[g];
    x = Group{0, 0, 0, 0, 0};
    if (b0 < 0 || b1 < b0 || b1 > a.num_seqs || S < 0 || S > a.max_shared_len) return false;
    const int c0 = a.cu_rows[b0], c1 = a.cu_rows[b1];
    if (c0 < 0 || c1 < c0 || c1 > a.total_rows || c1 - c0 > a.max_rows) return false;
    x = Group{b0, b1, c0, c1 - c0, S & ~(kBlock - 1)};
    return true;
}

// The shared positions of sequence b, in whole blocks, and its group (-1: none).
__device__ __forceinline__ int shared_of(const GroupArgs& a, int b, int& g) {
    int lo = 0, hi = a.num;  // the last group that begins at or before b
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.starts[mid] <= b) lo = mid; else hi = mid;
    }
    g = -1;
    Group x;
    if (!group_at(a, lo, x) || b < x.first || b >= x.last || x.shared == 0) return 0;
    g = lo;
    return x.shared;
}

}  // namespace msa
