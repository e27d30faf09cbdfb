// relative_bias.cu - buckets of a learned relative position bias, and its table by distance.
//
// A distance n = query position - key position >= 0 has bucket n below m = num_buckets / 2, and
// beyond it min(num_buckets - 1, m + floor(ln(n / m) / ln(max_distance / m) (num_buckets - m))).
// The floor is that of the real number: bucket m + j begins at the smallest n with
//     n^r >= m^(r - j) max_distance^j,   r = num_buckets - m,
// which is found in double precision and, where the border is next to a whole number, decided
// in whole numbers.
#include <math.h>

#include "pa_common.cuh"
#include "relative_bias.cuh"

namespace pa {

namespace {

// A whole number below 2^1152, least significant word first: n^r for distances below 2^16 and at most 64
// factors.
struct Whole {
    uint32_t w[36] = {1u};
    void multiply(uint32_t f) {
        uint64_t carry = 0;
        for (uint32_t &x : w) {
            carry += static_cast<uint64_t>(x) * f;
            x = static_cast<uint32_t>(carry);
            carry >>= 32;
        }
    }
};
static_assert(kMaxBuckets - kMaxBuckets / 2 <= 64 && kMaxBiasDistance < 1 << 16, "powers fit in a Whole");

// n^r >= m^(r - j) d^j
bool reaches(int n, int m, int d, int r, int j) {
    Whole a, b;
    for (int i = 0; i < r; ++i) {
        a.multiply(n);
        b.multiply(i < j ? d : m);
    }
    for (int i = 35; i >= 0; --i)
        if (a.w[i] != b.w[i]) return a.w[i] > b.w[i];
    return true;
}

// One thread an entry; a bucket's first distances are read through the kernel's parameters.  2 us for 32
// heads, 32 buckets to 128 (a launch's latency); a table by distance costs the attention kernels one read
// an element where the bucket's search would take five steps.
__global__ void __launch_bounds__(128)
    bias_table_kernel(float *__restrict__ table, const __grid_constant__ RelativeBias b, int num_heads) {
    bias_table_entry(table, b, num_heads, blockIdx.x * 128 + threadIdx.x, blockIdx.y, gridDim.y, num_heads);
}

}  // namespace

bool plan_relative_bias(int num_buckets, int max_distance, RelativeBias *b) {
    if (num_buckets < 2 || num_buckets > kMaxBuckets) return false;
    const int m = num_buckets / 2, r = num_buckets - m;
    if (max_distance <= m || max_distance > kMaxBiasDistance) return false;
    b->num_buckets = num_buckets;
    for (int i = 0; i <= m; ++i) b->first[i] = i;
    for (int j = 1; j < r; ++j) {
        const double x = m * pow(static_cast<double>(max_distance) / m, static_cast<double>(j) / r);
        const double whole = nearbyint(x);
        int n = static_cast<int>(ceil(x));
        // pow is within a few units of its last place; distances are below 2^15.
        if (fabs(x - whole) < 1e-9 * x) {
            n = static_cast<int>(whole);
            if (!reaches(n, m, max_distance, r, j)) ++n;
        }
        b->first[m + j] = n;
    }
    b->first[num_buckets] = 1 << 30;
    return true;
}

size_t bias_table_bytes(int num_heads, const RelativeBias &b) {
    return (static_cast<size_t>(num_heads) * bias_stride(b.last()) * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_bias_table(float *table, int num_heads, const RelativeBias &b, cudaStream_t stream) {
    const dim3 grid((bias_stride(b.last()) + 127) / 128, num_heads < 64 ? num_heads : 64);
    bias_table_kernel<<<grid, 128, 0, stream>>>(table, b, num_heads);
    return cudaGetLastError();
}

}  // namespace pa
