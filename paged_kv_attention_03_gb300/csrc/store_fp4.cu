// store_fp4.cu - the 4-bit cache's store (quantise and scatter) and its inverse (gather and
// expand).
//
// store:  for every token t with s = slot_mapping[t] >= 0, the K and V rows of t are quantised
//         group by group (fp4.cuh) into row (s / block_size, head, s % block_size).
// gather: key[t] = bf16(code * scale * kv_scale) of the row of slot_mapping[t]; zeros for a
//         negative slot.
//
// Both are HBM streams: a token and head is 4 D bytes of bf16 and 2 x 9/16 D bytes of cache.
// One thread takes one group of 16 dims of K and of V (32 bytes each of bf16, 8 bytes of
// codes): the groups of a row sit in consecutive lanes, so a row is written as one contiguous
// run, its scales gathered by shuffles and written by the row's first lane.
//
// Measured on 17403 tokens of 8 heads of 128 (91 MB each), three sets of tensors in turn: store
// 17.5 us (5.2 TB/s; issue slots 68 % busy, DRAM 46 %: neither at its limit, a thread loads,
// quantises and stores one group of K and V in that order), gather 16.4 us (5.6 TB/s).
#include "fp4.cuh"
#include "pa_internal.h"
#include "sm100_ptx.cuh"

namespace pa {

namespace {


// Cache row of (slot, head): [num_blocks, num_kv_heads, block_size] rows.
__device__ __forceinline__ int64_t cache_row(int64_t slot, int head, int kv_heads, int log2_bs) {
    return (((slot >> log2_bs) * kv_heads + head) << log2_bs) + (slot & ((1 << log2_bs) - 1));
}

// The place of group i: token, head, group of 16 dims (32-bit divisions where they do).
struct Place {
    int64_t token;
    int head;
    int group;
};
template <int GROUPS>
__device__ __forceinline__ Place place_of(int64_t i, int64_t total, int kv_heads) {
    if (total <= 0xffffffffll) {
        const unsigned th = static_cast<unsigned>(i) / GROUPS;
        const unsigned t = th / static_cast<unsigned>(kv_heads);
        return {t, static_cast<int>(th - t * kv_heads), static_cast<int>(i % GROUPS)};
    }
    const int64_t th = i / GROUPS;
    const int64_t t = th / kv_heads;
    return {t, static_cast<int>(th - t * kv_heads), static_cast<int>(i % GROUPS)};
}

__device__ __forceinline__ void load_words(const uint4 *src, uint32_t (&w)[8]) {
    const uint4 a = __ldcs(src), b = __ldcs(src + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// The scale codes of a row's D / 16 lanes as words of four, in the row's first lane.
template <int GROUPS>
__device__ __forceinline__ uint2 row_scales(uint32_t code, int g, unsigned mask) {
    uint32_t w = code << (8 * (g & 3));
    w |= __shfl_xor_sync(mask, w, 1);
    w |= __shfl_xor_sync(mask, w, 2);
    uint2 r = make_uint2(w, 0u);
    if constexpr (GROUPS == 8) r.y = __shfl_xor_sync(mask, w, 4);
    return r;
}

template <int D>
__device__ __forceinline__ void write_row(uint8_t *row, int g, uint2 codes, uint2 scales) {
    if constexpr (D == 128) {  // 72-byte rows: 8-byte aligned
        *reinterpret_cast<uint2 *>(row + 8 * g) = codes;
        if (g == 0) *reinterpret_cast<uint2 *>(row + 64) = scales;
    } else {  // 36-byte rows: 4-byte aligned
        uint32_t *r = reinterpret_cast<uint32_t *>(row);
        r[2 * g] = codes.x;
        r[2 * g + 1] = codes.y;
        if (g == 0) r[8] = scales.x;
    }
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(256)
store_kvcache_fp4_kernel(const uint4 *__restrict__ key, const uint4 *__restrict__ value,
                         uint8_t *__restrict__ k_cache, uint8_t *__restrict__ v_cache,
                         const int32_t *__restrict__ slot_mapping, int64_t total,
                         int64_t num_slots, int kv_heads, int log2_bs, float kv_scale,
                         float kv_scale6, unsigned *err) {
    constexpr int GROUPS = D / 16;
    constexpr int RB = fp4::row_bytes(D);
    const int lane = threadIdx.x & 31;
    // The lanes of one row: they take every branch together.
    const unsigned mask = ((1u << GROUPS) - 1u) << (lane & ~(GROUPS - 1));
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= total) return;
    const Place at = place_of<GROUPS>(i, total, kv_heads);
    const int g = at.group, h = at.head;
    const int64_t slot = __ldg(slot_mapping + at.token);
    if (slot < 0) return;  // padding token
    if (slot >= num_slots) {
        if (g == 0 && h == 0) flag_error(err, kErrSlotRange);
        return;
    }
    uint32_t kw[8], vw[8];
    load_words(key + 2 * i, kw);
    load_words(value + 2 * i, vw);
    uint32_t ks, vs;
    const uint2 kc = fp4::quant_group(kw, kv_scale, kv_scale6, ks);
    const uint2 vc = fp4::quant_group(vw, kv_scale, kv_scale6, vs);
    const uint2 kss = row_scales<GROUPS>(ks, g, mask), vss = row_scales<GROUPS>(vs, g, mask);
    const int64_t row = cache_row(slot, h, kv_heads, log2_bs);
    write_row<D>(k_cache + row * RB, g, kc, kss);
    write_row<D>(v_cache + row * RB, g, vc, vss);
}

namespace {

// One group of a row as 16 bf16 (32 bytes: one store where dst is aligned to that, so that the L2
// gets whole sectors).
template <int D, bool ALIGNED>
__device__ __forceinline__ void expand_group(const uint8_t *row, int g, float kv_scale, uint4 *dst) {
    uint32_t c[2];
    if constexpr (D == 128) {
        const uint2 v = *reinterpret_cast<const uint2 *>(row + 8 * g);
        c[0] = v.x;
        c[1] = v.y;
    } else {
        const uint32_t *r = reinterpret_cast<const uint32_t *>(row);
        c[0] = r[2 * g];
        c[1] = r[2 * g + 1];
    }
    const float s = fp4::f16_lo(fp4::e4m3x2_to_f16x2(row[D / 2 + g]));
    uint32_t o[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t f[4];
        fp4::e2m1x8_to_f16x2x4(c[h], f);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // code * scale is exact in fp32 too
            o[4 * h + k] = pack_bf16x2(fp4::f16_lo(f[k]) * s * kv_scale,
                                       fp4::f16_hi(f[k]) * s * kv_scale);
    }
    if constexpr (ALIGNED) {
        sm100::st_global_v8(dst, o);
    } else {
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace

template <int D, bool ALIGNED>
__global__ void __launch_bounds__(256)
gather_kvcache_fp4_kernel(uint4 *__restrict__ key, uint4 *__restrict__ value,
                          const uint8_t *__restrict__ k_cache, const uint8_t *__restrict__ v_cache,
                          const int32_t *__restrict__ slot_mapping, int64_t total,
                          int64_t num_slots, int kv_heads, int log2_bs, float kv_scale,
                          unsigned *err) {
    constexpr int GROUPS = D / 16;
    constexpr int RB = fp4::row_bytes(D);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= total) return;
    const Place at = place_of<GROUPS>(i, total, kv_heads);
    const int g = at.group, h = at.head;
    const int64_t slot = __ldg(slot_mapping + at.token);
    if (slot < 0 || slot >= num_slots) {
        if (slot >= 0 && g == 0 && h == 0) flag_error(err, kErrSlotRange);
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        key[2 * i] = z;
        key[2 * i + 1] = z;
        value[2 * i] = z;
        value[2 * i + 1] = z;
        return;
    }
    const int64_t row = cache_row(slot, h, kv_heads, log2_bs);
    expand_group<D, ALIGNED>(k_cache + row * RB, g, kv_scale, key + 2 * i);
    expand_group<D, ALIGNED>(v_cache + row * RB, g, kv_scale, value + 2 * i);
}

namespace {

constexpr int64_t kMostGroups = 0x7fffffffll * 256;  // one block for 256 groups

unsigned fp4_blocks(int64_t total) {
    return static_cast<unsigned>((total + 255) / 256);  // (checked against the grid's limit)
}

template <int D>
cudaError_t launch_store_d(const StoreArgs &a, int kv_heads, int log2_bs, float kv_scale,
                           cudaStream_t stream) {
    const int64_t total = a.num_tokens * kv_heads * (D / 16);
    store_kvcache_fp4_kernel<D><<<fp4_blocks(total), 256, 0, stream>>>(
        static_cast<const uint4 *>(a.key), static_cast<const uint4 *>(a.value),
        static_cast<uint8_t *>(a.k_cache), static_cast<uint8_t *>(a.v_cache), a.slot_mapping, total,
        a.num_slots, kv_heads, log2_bs, kv_scale, 6.f * kv_scale, a.err);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_gather_d(const GatherArgs &a, cudaStream_t stream) {
    const int64_t total = a.num_tokens * a.num_kv_heads * (D / 16);
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.key) | reinterpret_cast<uintptr_t>(a.value)) & 31u) == 0;
    auto kern = aligned ? gather_kvcache_fp4_kernel<D, true> : gather_kvcache_fp4_kernel<D, false>;
    kern<<<fp4_blocks(total), 256, 0, stream>>>(
        static_cast<uint4 *>(a.key), static_cast<uint4 *>(a.value),
        static_cast<const uint8_t *>(a.k_cache), static_cast<const uint8_t *>(a.v_cache),
        a.slot_mapping, total, a.num_slots, a.num_kv_heads, a.log2_bs, a.kv_scale, a.err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_store_kvcache_fp4(const StoreArgs &a, int kv_heads, int head_dim, int log2_bs,
                                     float kv_scale, cudaStream_t stream) {
    if (a.num_tokens == 0) return cudaSuccess;
    if (a.num_tokens > kMostGroups / (static_cast<int64_t>(kv_heads) * (head_dim / 16))) return cudaErrorInvalidValue;
    switch (head_dim) {
        case 64: return launch_store_d<64>(a, kv_heads, log2_bs, kv_scale, stream);
        case 128: return launch_store_d<128>(a, kv_heads, log2_bs, kv_scale, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_gather_kvcache_fp4(const GatherArgs &a, cudaStream_t stream) {
    if (a.num_tokens == 0) return cudaSuccess;
    if (a.num_tokens > kMostGroups / (static_cast<int64_t>(a.num_kv_heads) * (a.head_dim / 16))) return cudaErrorInvalidValue;
    switch (a.head_dim) {
        case 64: return launch_gather_d<64>(a, stream);
        case 128: return launch_gather_d<128>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
