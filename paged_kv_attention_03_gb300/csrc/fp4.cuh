// fp4.cuh - the 4-bit KV cache's number format and row layout.
//
// A cache row (one token of one kv head) is D / 2 bytes of E2M1 codes, two to a byte with
// the even head dim in the low four bits, then D / 16 E4M3 scales, one for each 16 dims:
//     element = code * scale * kv_scale.
// Every code * scale is an f16: E2M1 has 2 significant bits and E4M3 4, so a product has at
// most 6; its magnitude is 0 or between 2^-10 and 2688.  Rows of consecutive tokens of one
// kv head are contiguous, so 16 tokens are 9 D bytes that one bulk copy moves.
#pragma once

#include <math.h>
#include <stdint.h>

#include "pa_common.cuh"

namespace pa {
namespace fp4 {

// Bytes of a cache row.
__host__ __device__ constexpr int row_bytes(int head_dim) { return head_dim / 2 + head_dim / 16; }

// The four code pairs of a word -> four f16x2 (low code in the low half).
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t w, uint32_t (&f)[4]) {
    asm("{\n"
        ".reg .b8 a, b, c, d;\n"
        "mov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n"
        "}\n"
        : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
        : "r"(w));
}

// Two E4M3 codes (the low 16 bits, low byte first) -> f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t h;
    asm("{\n"
        ".reg .b16 a, b;\n"
        "mov.b32 {a, b}, %1;\n"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n"
        "}\n"
        : "=r"(h)
        : "r"(w));
    return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float f16_lo(uint32_t h) {
    float f;
    asm("{\n.reg .b16 l, u;\nmov.b32 {l, u}, %1;\ncvt.f32.f16 %0, l;\n}\n" : "=f"(f) : "r"(h));
    return f;
}
__device__ __forceinline__ float f16_hi(uint32_t h) { return f16_lo(h >> 16); }

// The smallest scale code a group gets (2^-9): a group of zeros needs no other case.
constexpr uint32_t kMinScale = 1;

// Quantise one group: 16 bf16 (8 words, low half first) -> 8 bytes of codes and a scale code.
//     scale = max(E4M3(max|x| / (6 kv_scale)), 2^-9),  code = E2M1(x / (scale * kv_scale)),
// each division and product one fp32 operation, each conversion to the nearest with ties to
// even, saturating (448, 6).  A NaN in the group makes its scale NaN, so the group reads NaN;
// an infinity saturates.
//
// The 16 quotients share their divisor d: with r the rounded reciprocal, q = x r and one
// correction q - (q d - x) r by two fused operations give the rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990, asks for
// a q within one unit; here every 8-bit x against every 24-bit d was tried, and all 2^30
// quotients are the rounded ones).  That scales by powers of two as long as q d - x keeps its
// bits, which kv_scale >= 1e-25 sees to.  Written this way round a zero keeps its sign: for
// x = -0 the remainder is (-0) - (-0) = +0 and the sum (-0) + (-0); x - q d would add +0.  17403 tokens: 18.3 us against 23.5 with divisions.
__device__ __forceinline__ uint2 quant_group(uint32_t (&w)[8], float kv_scale, float kv_scale6,
                                             uint32_t &scale_code) {
    // Magnitudes of bf16 order like their bit patterns, and a NaN's is above infinity's.
    uint32_t top = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    const float amax = __uint_as_float(max(top & 0xffffu, top >> 16) << 16);
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(s8)
        : "f"(0.f), "f"(__fdiv_rn(amax, kv_scale6)));
    scale_code = max(static_cast<uint32_t>(s8) & 0xffu, kMinScale);
    const float den = __fmul_rn(f16_lo(e4m3x2_to_f16x2(scale_code)), kv_scale);
    const float r = __frcp_rn(den);
    if (scale_code >= 126u) {
        // Only a saturated scale leaves quotients beyond 9 (the smallest scales are coarse: 2^-9
        // stands for up to 1.5 times itself), up to infinity: those saturate too.
        const __nv_bfloat162 most = __float2bfloat162_rn(8.f * den);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 x = __hmax2(__hmin2(*reinterpret_cast<__nv_bfloat162 *>(&w[i]), most), __hneg2(most));
            w[i] = *reinterpret_cast<const uint32_t *>(&x);
        }
    }
    auto quotient = [&](float x) {
        const float q = __fmul_rn(x, r);
        return __fmaf_rn(-__fmaf_rn(q, den, -x), r, q);
    };
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float lo = quotient(__uint_as_float(w[i] << 16));
        const float hi = quotient(__uint_as_float(w[i] & 0xffff0000u));
        uint32_t b;
        asm("{\n.reg .b8 t;\ncvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\ncvt.u32.u8 %0, t;\n}\n"
            : "=r"(b)
            : "f"(hi), "f"(lo));
        c[i >> 2] |= b << (8 * (i & 3));
    }
    return make_uint2(c[0], c[1]);
}

}  // namespace fp4
}  // namespace pa
