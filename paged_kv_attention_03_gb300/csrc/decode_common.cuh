// decode_common.cuh - device helpers shared by the decode kernels (decode.cu, decode_fp4.cu).
#pragma once

#include <stdint.h>

#include "pa_common.cuh"

namespace pa {

// Key range of one sequence: keys [start, L); splits tile [base, L) in `chunk`s.
struct SeqRange {
    int L;
    int start;
    int base;
};

__device__ __forceinline__ SeqRange decode_range(int raw_len, int64_t cap, int window,
                                                 int key_begin, unsigned *err, bool report) {
    SeqRange r;
    int L = raw_len;
    if (L < 0 || static_cast<int64_t>(L) > cap) {
        if (report) flag_error(err, kErrSeqRange);
        L = L < 0 ? 0 : static_cast<int>(cap);
    }
    r.L = L;
    r.start = window > 0 ? max(0, L - window) : 0;
    if (key_begin > r.start) r.start = min(key_begin, L);  // partial state from key_begin
    r.base = r.start & ~15;
    return r;
}

// Transpose of an 8x8 matrix of 16-bit elements held as the MMA accumulator fragment
// (lane holds row lane/4, columns 2 (lane%4) and + 1): afterwards the lane holds row
// lane/4 of the transpose.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4],
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace pa
