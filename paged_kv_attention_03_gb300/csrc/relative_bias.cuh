// relative_bias.cuh - the table of a learned relative position bias by distance.
//
// Row h holds head h's bias times log2(e) for the distances -kBiasPad .. last + kBiasTail - 1 (last:
// the first distance of the last bucket).  Entries below 0 are -inf, which hides future keys, and those
// from last on are all the last bucket's, so that a kernel may read whole runs around a tile's
// distances without clamping each one.
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int kBiasPad = 256, kBiasTail = 128;

__host__ __device__ inline int bias_stride(int last) { return (last + kBiasPad + kBiasTail + 3) & ~3; }

// Entry of distance 0 of a head's row.
__device__ __forceinline__ const float *bias_row_of(const float *table, int head, int last) {
    return table + static_cast<int64_t>(head) * bias_stride(last) + kBiasPad;
}

// The bucket of distance n >= 0: the last one that begins at n or before.
__device__ __forceinline__ int bucket_of(const RelativeBias &b, int n) {
    int lo = 0, hi = b.num_buckets;  // first[lo] <= n < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.first[mid] <= n)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

}  // namespace pa
