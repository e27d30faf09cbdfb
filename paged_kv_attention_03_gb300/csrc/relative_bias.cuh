// relative_bias.cuh - the table of a learned relative position bias by distance.
//
// Row h holds head h's bias in base-2 units (times log2 e) for the distances 0 .. last + kBiasTail - 1
// (last: the first distance of the last bucket), less bias_ref.  Entries before distance 0 are -inf, which
// hides future keys; those from last on are all the last bucket's.  So a kernel may read whole runs
// around a tile's distances without clamping each one.
#pragma once

#include <math.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

// (Both cover a prefill item's tile: 256 tokens against 128 keys.)
constexpr int kBiasPad = 384, kBiasTail = 392;  // (entries before distance 0, and from last on)

__host__ __device__ inline int bias_stride(int last) { return (last + kBiasPad + kBiasTail + 3) & ~3; }

// A bias in base-2 units.  What lies below -1e30 hides its keys as -inf does: a row that saw nothing else
// would have a log-sum-exp whose last place is larger than any logit.
__device__ __forceinline__ float bias_log2(float b) { return b < -1e30f ? -INFINITY : b * kLog2e; }

// Entries are what is left over bias_ref, which is the last bucket's bias unless that is so large that the
// difference would lose the others' digits; then far keys' logits need no change of their own.  A row's
// first entry is the last bucket's bias itself.
__device__ __forceinline__ float bias_ref(float far) { return fabsf(far) <= 64.f ? far : 0.f; }

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

// Entry i of the rows of heads h, h + step, ... below end.  (The heads share the search.)
__device__ __forceinline__ void bias_table_entry(float *__restrict__ table, const RelativeBias &b, int num_heads, int i, int h, int step,
                                                 int end) {
    const int stride = bias_stride(b.last());
    if (i >= stride) return;
    const int k = bucket_of(b, max(i - kBiasPad, 0));
    for (; h < end; h += step) {
        const float far = bias_log2(b.bias[static_cast<int64_t>(b.num_buckets - 1) * num_heads + h]);
        const float v = bias_log2(b.bias[static_cast<int64_t>(k) * num_heads + h]);
        table[static_cast<int64_t>(h) * stride + i] = i == 0 ? far : i < kBiasPad ? -INFINITY : v - bias_ref(far);
    }
}

}  // namespace pa
