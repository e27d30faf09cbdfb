// attn_backward.cu - gradient of packed variable-length attention on the sm_103a tensor cores
// (tcgen05 + TMEM).
//
// With s_ij = scale q_i k_j + bias(p_i - j), P_ij = e^(s_ij - lse_i) over the keys j that row i sees,
// out = P V and dout given:
//     dP = dout V^T,   D_i = sum_j P_ij dP_ij,   dS = P (dP - D),
//     dV = P^T dout,   dQ = scale dS K,   dK = scale dS^T Q,   dbias_b = sum of dS over bucket b.
// D_i also equals dout_i out_i, but out is bf16 there: good enough inside dQ, whose terms are rounded
// to bf16 anyway, unless a row's dS nearly cancel, as they do in rows of few keys; and not for sums
// of dS.  So the dQ kernel starts from dout_i out_i, goes twice over the tiles that need the sum
// itself, first for D alone, and leaves D in fp32 for dK.
//
// Two kernels share the work, each with its accumulators in tensor memory and no atomics, so equal
// calls give equal bits:
//  * grad_q_kernel: 128 queries of one head against their keys in turn (3 products a tile).  dbias: the
//    tiles whose distances all belong to the last bucket add sum_j P dP - D sum_j P to it; the others,
//    the nearest ones, come last, once for D and once more with it, and their dS are summed along
//    diagonals into buckets;
//  * grad_kv_kernel: 128 keys of one kv head against the queries of every head that shares it
//    (4 products a tile), so the sum over the heads happens in the accumulator;
// The products count 7 for the 5 of the formula (S and dP are formed twice); dQ added up across
// the CTAs of one pass over the keys would need atomics, whose order changes the result.
//
// Roles in a CTA: warps 0-7 are two warpgroups of element-wise work, each on 64 of a tile's 128
// columns (a thread owns a TMEM lane, i.e. an accumulator row); warp 8 loads tiles by TMA, warp 9
// issues the products.  P and dS go back to tensor memory as bf16, over the fp32 tile they came
// from, and are the first operand of the next product from there.
#include <cuda.h>

#include <atomic>
#include <climits>
#include <cstring>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "relative_bias.cuh"
#include "sm100_ptx.cuh"

namespace pa {

namespace {

using namespace sm100;

constexpr int BM = 128;                 // rows (TMEM lanes) of a tile
constexpr int BN = 128;                 // columns of a tile
constexpr uint32_t HALF = 128u * 128u;  // [128 rows][64 bf16]: one swizzle span
constexpr int kWarpLoad = 8, kWarpMma = 9;
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;
// Rows of fewer keys get their D from the sum over the keys also for dQ.  dout . out is off by about
// 2^-9 |dout . out|, and |dout . out| shrinks against dP as the root of the number of keys that share
// the weight: from 128 on the error is below a tenth of that of dS in bf16.
constexpr int kFewKeys = 128;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per wait

struct GradParams {
    // Boxes of 64 dims of one head: [0] of 128 rows, [1] of 16 rows.
    CUtensorMap tmap_q[2];
    CUtensorMap tmap_do[2];
    CUtensorMap tmap_k[2];
    CUtensorMap tmap_v[2];
    const int32_t *cu_q;
    const int32_t *cu_k;
    __nv_bfloat16 *dq;
    __nv_bfloat16 *dk;
    __nv_bfloat16 *dv;
    int64_t dq_stride, dk_stride, dv_stride;
    const float *lse2;  // [num_heads, total_q]: lse in base 2, +inf for a row without keys
    float *delta;       // [num_heads, total_q]: D
    const float *bias_table;
    float *partial;     // [slots, num_heads, num_buckets]
    int num_seqs;
    int total_q, total_k;
    int max_q, max_k;
    int q_tiles;
    int num_heads, num_kv_heads, group;
    int window;
    float scale, scale_log2;
    unsigned *err;
    RelativeBias bias;
};

struct Seq {
    int q_start, sq, k_start, sk;
    bool ok;
};

__device__ __forceinline__ Seq load_seq(const GradParams &p, int seq, bool report) {
    Seq s;
    s.q_start = p.cu_q[seq];
    s.sq = p.cu_q[seq + 1] - s.q_start;
    s.k_start = p.cu_k[seq];
    s.sk = p.cu_k[seq + 1] - s.k_start;
    const bool q_ok = s.q_start >= 0 && s.sq >= 0 && static_cast<int64_t>(s.q_start) + s.sq <= p.total_q && s.sq <= p.max_q;
    const bool k_ok = s.k_start >= 0 && s.sk >= 0 && static_cast<int64_t>(s.k_start) + s.sk <= p.total_k && s.sk <= p.max_k;
    if (report && !q_ok) flag_error(p.err, kErrQueryLen);
    if (report && !k_ok) flag_error(p.err, kErrSeqRange);
    s.ok = q_ok && k_ok;
    return s;
}

// Shared memory: two resident tiles (Q and dout, or K and V), rings of the tiles that pass by (K
// and V, or Q and dout), small arrays, barriers.  K outlives V by the time from dP to dQ, so it has
// three stages there.
template <int HD, int STAGES_A, uint32_t SMALL_BYTES>
struct Layout {
    static constexpr int NHALF = HD / 64;
    static constexpr uint32_t TILE = NHALF * HALF;
    static constexpr int NA = STAGES_A, NB = 2;
    static constexpr uint32_t OFF_RES = 0;
    static constexpr uint32_t OFF_A = 2 * TILE;          // Q (dK, dV) or K (dQ)
    static constexpr uint32_t OFF_B = OFF_A + NA * TILE;  // dout (dK, dV) or V (dQ)
    static constexpr uint32_t OFF_SMALL = OFF_B + NB * TILE;
    static constexpr uint32_t OFF_BAR = OFF_SMALL + SMALL_BYTES;
    static constexpr uint32_t OFF_MISC = OFF_BAR + 160;
    static constexpr uint32_t BYTES = OFF_MISC + 16;
    // At least 116 KB so a single CTA owns an SM (and all of its TMEM).
    static constexpr uint32_t SMEM = (BYTES > 118784u ? BYTES : 118784u);
    static_assert(SMEM <= 232448u, "at most 227 KB of shared memory per CTA");
};

template <int HD>
using LayoutQ = Layout<HD, 3, 2048>;
template <int HD>
using LayoutKv = Layout<HD, 2, 2u * 3 * 512>;

enum : int {
    B_RES = 0,      // resident tiles loaded
    B_AFULL = 1,    // [3] tile of ring A ready (two arrivals: the copies, and the loading warp)
    B_AEMPTY = 4,   // [3] read
    B_BFULL = 7,    // [2] ring B, likewise
    B_BEMPTY = 9,   // [2]
    B_LAND = 11,    // copies of a tile that the loading warp edits
    B_SFULL = 12,   // logits of a tile ready
    B_PFULL = 13,   // logits read (dQ), or P in tensor memory (dK, dV) (8 warps)
    B_DPFULL = 14,  // [2] dP ready
    B_DSFULL = 16,  // [2] dS in tensor memory (8 warps)
    B_DONE = 18,    // all products done
    B_SUMS = 19,    // both halves of the rows' D written (8 warps)
    NBARS = 20
};

// A [128][HD] tile from row0 of a sequence that ends at row `end`: a box a lane.  A tile that the
// sequence fills comes in boxes of 128 rows (a pair of tiles in 16-row pieces took 2900 cycles to land,
// 1400 this way), another one in 16-row pieces, those past the end from an out-of-range row, which
// reads as zeros.
template <int HD>
__device__ __forceinline__ void load_tile(const CUtensorMap *map, uint32_t dst, int head, int start, int row0, int end,
                                          uint32_t bar) {
    constexpr int NHALF = HD / 64;
    const int lane = threadIdx.x & 31;
    if (end - row0 >= BM) {
        if (lane < NHALF) tma_load_3d(dst + lane * HALF, map, lane * 64, head, start + row0, bar);
    } else if (lane < 8 * NHALF) {
        const int u = lane / NHALF, h = lane - u * NHALF;
        const int row = row0 + 16 * u < end ? start + row0 + 16 * u : -16;
        tma_load_3d(dst + h * HALF + u * 2048, map + 1, h * 64, head, row, bar);
    }
}

// Rows `from` .. of the last 16-row piece belong to the next sequence: zeros, so that a product over
// rows gets nothing from them whatever they hold.
template <int HD>
__device__ __forceinline__ void clear_rows(uint32_t tile, int from) {
    constexpr int NHALF = HD / 64;
    const int rows = 16 - (from & 15);
    for (int i = threadIdx.x & 31; i < rows * 8 * NHALF; i += 32) {
        const int r = from + i / (8 * NHALF), c = i % (8 * NHALF);
        st_shared_v4(tile + (c >> 3) * HALF + r * 128 + (c & 7) * 16, 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
}
__device__ __forceinline__ bool ragged(int left) { return left < BM && (left & 15) != 0; }

// Tile -> stage, by the loading warp; `full` expects two arrivals.  `lands` counts the edited tiles,
// `extra` runs before the second arrival.  False: a wait ran out.
template <int HD, class Extra>
__device__ __forceinline__ bool load_stage(const CUtensorMap *map, uint32_t dst, int head, int start, int row0, int end,
                                           uint32_t full, uint32_t land, uint32_t &lands, volatile int *abort_flag,
                                           unsigned *err, Extra extra) {
    const int lane = threadIdx.x & 31;
    const bool cut = ragged(end - row0);
    if (lane == 0) mbar_arrive_expect_tx(cut ? land : full, (HD / 64) * HALF);
    __syncwarp();
    load_tile<HD>(map, dst, head, start, row0, end, cut ? land : full);
    extra();
    if (cut) {
        if (!wait_warp(land, lands++ & 1, abort_flag, err, kTimeoutNs)) return false;
        clear_rows<HD>(dst, end - row0);
    }
    __syncwarp();
    if (lane == 0) {
        if (cut) mbar_arrive(full);
        mbar_arrive(full);
    }
    return true;
}

// D[128 x 128] = A B^T over HD dims, both tiles [128][HD].
template <int HD>
__device__ __forceinline__ void issue_abt(uint32_t d, uint32_t a, uint32_t b) {
    constexpr uint32_t idesc = idesc_bf16_f32(BM, BN, false);
    const uint64_t a0 = smem_desc_sw128(a, 16, 1024), b0 = smem_desc_sw128(b, 16, 1024);
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
        const uint32_t off = (k >> 2) * HALF + (k & 3) * 32;
        mma_bf16_ss(d, desc_advance(a0, off), desc_advance(b0, off), idesc, k > 0);
    }
}

// D[128 x HD] += A B: A [128 x 128] bf16 in tensor memory (columns 0-31 hold its first 64 columns,
// 64-95 the others: each warpgroup wrote over its own half), B a [128][HD] tile.
template <int HD>
__device__ __forceinline__ void issue_ab(uint32_t d, uint32_t a, uint32_t b, bool first) {
    constexpr uint32_t idesc = idesc_bf16_f32(BM, HD, true);
    const uint64_t b0 = smem_desc_sw128(b, HALF, 1024);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        mma_bf16_ts(d, a + (k & 3) * 8 + (k >> 2) * 64, desc_advance(b0, k * 2048), idesc, (!first || k > 0) ? 1u : 0u);
}

// 32 columns of accumulator row `taddr` times f as bf16.
__device__ __forceinline__ void store_chunk(uint32_t taddr, float f, __nv_bfloat16 *dst, bool valid, bool v8) {
    float o[32];
    tmem_ld_32x32b_x32(taddr, o);
    tmem_wait_ld_regs(o);
    if (!valid) return;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(o[2 * i] * f, o[2 * i + 1] * f);
    if (v8) {
        st_global_v8(dst, w);
        st_global_v8(dst + 16, w + 8);
    } else {
        uint4 *d4 = reinterpret_cast<uint4 *>(dst);
#pragma unroll
        for (int i = 0; i < 4; ++i) d4[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}
__device__ __forceinline__ bool aligned32(const void *ptr, int64_t stride) {
    return ((reinterpret_cast<uintptr_t>(ptr) | static_cast<uintptr_t>(stride * 2)) & 31u) == 0;
}
template <int HD>
__device__ __forceinline__ void zero_rows(__nv_bfloat16 *dst, int64_t stride, int rows) {
    for (int i = threadIdx.x; i < rows * (HD / 8); i += kThreads)
        *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(i / (HD / 8)) * stride + i % (HD / 8) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
}

// Shared set-up of both kernels.
struct Cta {
    uint32_t base;
    uint8_t *sb;
    uint32_t tmem;
    volatile int *abort_flag;
};
template <class L>
__device__ __forceinline__ Cta setup() {
    extern __shared__ __align__(1024) uint8_t smem_raw[];  // (swizzled tiles start on 1024 bytes)
    Cta c;
    c.base = smem_u32(smem_raw);
    c.sb = smem_raw;
    c.abort_flag = reinterpret_cast<volatile int *>(c.sb + L::OFF_MISC + 4);
    auto bar = [&](int i) -> uint32_t { return c.base + L::OFF_BAR + 8u * static_cast<uint32_t>(i); };
    if (threadIdx.x == 0) {
        mbar_init(bar(B_RES), 1);
        for (int s = 0; s < 3; ++s) {
            mbar_init(bar(B_AFULL + s), 2);
            mbar_init(bar(B_AEMPTY + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(B_BFULL + s), 2);
            mbar_init(bar(B_BEMPTY + s), 1);
            mbar_init(bar(B_DPFULL + s), 1);
            mbar_init(bar(B_DSFULL + s), 8);
        }
        mbar_init(bar(B_LAND), 1);
        mbar_init(bar(B_SFULL), 1);
        mbar_init(bar(B_PFULL), 8);
        mbar_init(bar(B_DONE), 1);
        mbar_init(bar(B_SUMS), 8);
        *c.abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if ((threadIdx.x >> 5) == kWarpMma) {
        tmem_alloc(c.base + L::OFF_MISC, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    c.tmem = *reinterpret_cast<volatile uint32_t *>(c.sb + L::OFF_MISC);
    return c;
}
__device__ __forceinline__ void teardown(const Cta &c) {
    tc_fence_before();
    __syncthreads();
    if (*c.abort_flag) {
        // Bounded drain: let products and copies still in flight land before this CTA's shared
        // and tensor memory are released.
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
        __syncthreads();
    }
    if ((threadIdx.x >> 5) == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(c.tmem, kTmemCols);
    }
}

// ------------------------------------------------------------- rows' statistics ---
// lse in base 2 and dout_i out_i, both as [num_heads, total_q].  A block takes 8 tokens of 8 heads:
// half a warp (128 dims) or a quarter (64) a row.
template <int HD>
__global__ void __launch_bounds__(256)
    grad_stat_kernel(const uint4 *__restrict__ out, const uint4 *__restrict__ dout, const float *__restrict__ lse,
                     float *__restrict__ lse2, float *__restrict__ delta, int total_q, int num_heads) {
    constexpr int LANES = HD / 8, ROWS = 256 / LANES;
    __shared__ float s_l[8][9], s_d[8][9];  // [head][token]
    const int t0 = blockIdx.x * 8, h0 = blockIdx.y * 8;
    const int l = threadIdx.x % LANES;
#pragma unroll
    for (int r = threadIdx.x / LANES; r < 64; r += ROWS) {
        const int t = t0 + r / 8, h = h0 + r % 8;
        float d = 0.f;
        const bool in = t < total_q && h < num_heads;
        const int64_t row = static_cast<int64_t>(t) * num_heads + h;
        if (in) {
            const uint4 a = out[row * LANES + l], b = dout[row * LANES + l];
            const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d += __uint_as_float(x[i] << 16) * __uint_as_float(y[i] << 16) +
                     __uint_as_float(x[i] & 0xffff0000u) * __uint_as_float(y[i] & 0xffff0000u);
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (l == 0 && in) {
            const float e = lse[row];
            s_l[r % 8][r / 8] = e == -INFINITY ? INFINITY : e * kLog2e;
            s_d[r % 8][r / 8] = d;
        }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        const int i = threadIdx.x & 63, h = h0 + i / 8, t = t0 + i % 8;
        if (h < num_heads && t < total_q) {
            const int64_t at = static_cast<int64_t>(h) * total_q + t;
            if (threadIdx.x < 64)
                lse2[at] = s_l[i / 8][i % 8];
            else
                delta[at] = s_d[i / 8][i % 8];
        }
    }
}

// ------------------------------------------------------------------------- dQ ---
// Tensor memory: S at 0, dP (then dS) of two tiles in turn at 128 and 256, dQ at 384.  S is free once
// its rows are in registers, so the products of the next tile run while this one's dS is formed:
//     S(j + 1), dP(j + 1), then dQ(j).
template <int HD, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) grad_q_kernel(const __grid_constant__ GradParams p) {
    using L = LayoutQ<HD>;
    constexpr int NA = L::NA;
    constexpr uint32_t kDp = 128, kDq = 384;
    const int h = blockIdx.x % p.num_heads;
    const int rest = blockIdx.x / p.num_heads;
    const int seq = rest % p.num_seqs;
    const int qt = p.q_tiles - 1 - rest / p.num_seqs;  // rows with more keys first
    const Seq s = load_seq(p, seq, h == 0 && qt == 0 && threadIdx.x == 0);
    const int r0 = qt * BM;
    if (!s.ok || r0 >= s.sq) return;
    const int rows = min(BM, s.sq - r0);
    const int p_lo = s.sk - s.sq + r0, p_hi = p_lo + rows - 1;  // positions
    const int kmin = p.window > 0 ? max(0, p_lo - p.window + 1) : 0;
    const int last = p.bias.last();
    const int kt0 = kmin / BN;
    const int n = p_hi < 0 ? 0 : p_hi / BN - kt0 + 1;
    // Steps: the tiles 0 .. n_pre - 1 with D from dout . out; tiles n_pre .. n - 1 for D alone; then the
    // same with D.
    const bool few = p_lo + 1 < kFewKeys || (p.window > 0 && p.window < kFewKeys);
    const int n_far = BIAS ? min(max(kmin, p_lo - last + 1) / BN - kt0, n) : n;  // tiles of the last bucket alone
    const int n_pre = few ? 0 : n_far;
    const int n_all = 2 * n - n_pre;
    auto tile_of = [&](int j) -> int { return j < n ? j : j - (n - n_pre); };
    const int64_t stat_row = static_cast<int64_t>(h) * p.total_q + s.q_start + r0;
    __nv_bfloat16 *dq = p.dq + (static_cast<int64_t>(s.q_start) + r0) * p.dq_stride + h * HD;
    if (n == 0) {
        zero_rows<HD>(dq, p.dq_stride, rows);
        for (int i = threadIdx.x; i < rows; i += kThreads) p.delta[stat_row + i] = 0.f;
        return;
    }
    const Cta c = setup<L>();
    auto bar = [&](int i) -> uint32_t { return c.base + L::OFF_BAR + 8u * static_cast<uint32_t>(i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sQ = c.base + L::OFF_RES, sDo = sQ + L::TILE;
    auto sK = [&](int st) -> uint32_t { return c.base + L::OFF_A + st * L::TILE; };
    auto sV = [&](int st) -> uint32_t { return c.base + L::OFF_B + st * L::TILE; };
    // The rows' half sums [2][128], the warps' runs of diagonals [8][32].
    float *small = reinterpret_cast<float *>(c.sb + L::OFF_SMALL);
    const int kvh = h / p.group;
    // What the element-wise warps have at the end.
    float d_sum = 0.f;
    [[maybe_unused]] float d_far = 0.f, w_far = 0.f;  // sums of P dP and of P over the first n_far tiles
    [[maybe_unused]] float by_bucket[4] = {0.f, 0.f, 0.f, 0.f};

    if (warp == kWarpLoad) {
        if (lane < 4) prefetch_tmap(lane == 0 ? p.tmap_q : lane == 1 ? p.tmap_do : lane == 2 ? p.tmap_k : p.tmap_v);
        uint32_t lands = 0;
        // (Sums along diagonals run across rows; in all else a row behind the sequence stays on its own.)
        const bool edit = BIAS && ragged(rows);
        if (lane == 0) mbar_arrive_expect_tx(bar(edit ? B_LAND : B_RES), 2 * L::TILE);
        __syncwarp();
        load_tile<HD>(p.tmap_q, sQ, h, s.q_start, r0, s.sq, bar(edit ? B_LAND : B_RES));
        load_tile<HD>(p.tmap_do, sDo, h, s.q_start, r0, s.sq, bar(edit ? B_LAND : B_RES));
        bool ok = true;
        if (edit) {
            ok = wait_warp(bar(B_LAND), lands++ & 1, c.abort_flag, p.err, kTimeoutNs);
            if (ok) {
                clear_rows<HD>(sQ, rows);
                clear_rows<HD>(sDo, rows);
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(bar(B_RES));
        }
        auto load = [&](const CUtensorMap *map, uint32_t dst, int j, uint32_t full) -> bool {
            return load_stage<HD>(map, dst, kvh, s.k_start, (kt0 + tile_of(j)) * BN, s.sk, full, bar(B_LAND), lands,
                                  c.abort_flag, p.err, [] {});
        };
        for (int j = 0; ok && j < n_all; ++j) {
            const int sa = j % NA, sb = j & 1;
            if (j >= NA && !wait_warp(bar(B_AEMPTY + sa), (j / NA - 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
            if (!load(p.tmap_k, sK(sa), j, bar(B_AFULL + sa))) break;
            if (j >= 2 && !wait_warp(bar(B_BEMPTY + sb), ((j >> 1) - 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
            ok = load(p.tmap_v, sV(sb), j, bar(B_BFULL + sb));
        }
    } else if (warp == kWarpMma) {
        if (lane == 0) {
            auto wait = [&](int b, uint32_t parity) { return wait1(bar(b), parity, c.abort_flag, p.err, kTimeoutNs); };
            auto products = [&](int j) -> bool {  // S(j) and dP(j)
                if (!wait(B_AFULL + j % NA, (j / NA) & 1)) return false;
                tc_fence_after();
                issue_abt<HD>(c.tmem, sQ, sK(j % NA));
                mma_commit(bar(B_SFULL));
                if (!wait(B_BFULL + (j & 1), (j >> 1) & 1)) return false;
                tc_fence_after();
                issue_abt<HD>(c.tmem + kDp + 128u * (j & 1), sDo, sV(j & 1));
                mma_commit(bar(B_DPFULL + (j & 1)));
                mma_commit(bar(B_BEMPTY + (j & 1)));
                return true;
            };
            bool ok = wait(B_RES, 0) && products(0);
            for (int j = 0; ok && j < n_all; ++j) {
                // (dP(j + 1) goes where dS(j - 1) was: dQ(j - 1) is before it in the queue.)
                if (j + 1 < n_all && !(wait(B_PFULL, j & 1) && products(j + 1))) break;
                ok = wait(B_DSFULL + (j & 1), (j >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                if (j < n_pre || j >= n)
                    issue_ab<HD>(c.tmem + kDq, c.tmem + kDp + 128u * (j & 1), sK(j % NA), j == (n_pre > 0 ? 0 : n));
                mma_commit(bar(B_AEMPTY + j % NA));
                if (j + 1 == n_all) mma_commit(bar(B_DONE));
            }
        }
    } else {
        const int wg = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
        const bool valid = row < rows;
        const float lse2 = valid ? p.lse2[stat_row + row] : INFINITY;
        float delta = valid ? p.delta[stat_row + row] : 0.f;
        const float sl2 = p.scale_log2;
        const int pos = p_lo + row;
        [[maybe_unused]] const float *bias_row = nullptr;
        float far = -lse2;  // x = sl2 s + far, where the bias is that of the last bucket
        if constexpr (BIAS) {
            bias_row = bias_row_of(p.bias_table, h, last);
            far = __ldg(bias_row + last) - lse2;
        }
        const uint64_t sl2x2 = f2_pack(sl2, sl2), far2 = f2_pack(far, far);
        for (int j = 0; j < n_all; ++j) {
            const uint32_t dp = c.tmem + t_lane + kDp + 128u * (j & 1) + 64u * wg;
            const bool sum_only = j >= n_pre && j < n;
            const int tile = tile_of(j);
            const int key0 = (kt0 + tile) * BN + 64 * wg;  // this warpgroup's first key
            if (!wait_warp(bar(B_SFULL), j & 1, c.abort_flag, p.err, kTimeoutNs)) break;
            tc_fence_after();
            float w[2][32];  // logits, then weights P
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) tmem_ld_32x32b_x32(c.tmem + t_lane + 64u * wg + 32u * cc, w[cc]);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) tmem_wait_ld_regs(w[cc]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_PFULL));
            const int d0 = pos - key0;  // distance to the first key
            bool near = false;
            if constexpr (BIAS) near = __shfl_sync(0xffffffffu, d0, 0) - 63 < last && __shfl_sync(0xffffffffu, d0, 31) >= 0;
            if (near) {
                const float *bt = bias_row + d0;
#pragma unroll
                for (int i = 0; i < 64; ++i) w[i >> 5][i & 31] = fmaf(w[i >> 5][i & 31], sl2, __ldg(bt - i)) - lse2;
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float &a = w[i >> 4][2 * (i & 15)], &b = w[i >> 4][2 * (i & 15) + 1];
                    f2_unpack(f2_fma(f2_pack(a, b), sl2x2, far2), a, b);
                }
            }
            if (d0 < 63) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i > d0) w[i >> 5][i & 31] = -INFINITY;
            }
            if (p.window > 0 && d0 >= p.window) {
                const int first = d0 - p.window + 1;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i < first) w[i >> 5][i & 31] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) w[i >> 5][i & 31] = ex2_approx(w[i >> 5][i & 31]);
            if (BIAS && !sum_only && tile < n_far) {
                float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 64; ++i) a[i & 3] += w[i >> 5][i & 31];
                w_far += (a[0] + a[1]) + (a[2] + a[3]);
            }
            if (!wait_warp(bar(B_DPFULL + (j & 1)), (j >> 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
            tc_fence_after();
            uint32_t pk[32];
            uint64_t acc[2] = {0ull, 0ull};
            const uint64_t delta2 = f2_pack(-delta, -delta);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                float d[32];
                tmem_ld_32x32b_x32(dp + 32u * cc, d);
                tmem_wait_ld_regs(d);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint64_t w2 = f2_pack(w[cc][2 * i], w[cc][2 * i + 1]), d2 = f2_pack(d[2 * i], d[2 * i + 1]);
                    acc[i & 1] = f2_fma(w2, d2, acc[i & 1]);
                    f2_unpack(f2_mul(w2, f2_add(d2, delta2)), w[cc][2 * i], w[cc][2 * i + 1]);
                    pk[16 * cc + i] = pack_bf16x2(w[cc][2 * i], w[cc][2 * i + 1]);
                }
            }
            float a0, a1;
            f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
            d_sum += a0 + a1;
            if (!sum_only) {
                if (BIAS && tile + 1 == n_far) d_far = d_sum;
                tmem_st_32x32b_x32_u(dp, pk);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DSFULL + (j & 1)));
            if (j + 1 == n && n_pre < n) {
                // D of the row: this warpgroup's half and the other's.
                small[128 * wg + row] = d_sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_SUMS));
                if (!wait_warp(bar(B_SUMS), 0, c.abort_flag, p.err, kTimeoutNs)) break;
                delta = small[row] + small[128 + row];
                if (few) d_sum = 0.f;  // (the sums of the last bucket's tiles are formed in the second round)
            }
            if (BIAS && j >= n && tile >= n_far) {
                // Sums along the diagonals row - column = lane, lane - 32, lane - 64 of the warp's 32 x
                // 64 block: at column i the lane fetches the element of row (lane + i) % 32.
                float a[3] = {0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const float v = __shfl_sync(0xffffffffu, w[i >> 5][i & 31], lane + i);
                    const bool wrap = lane + (i & 31) >= 32;
                    if (wrap)
                        a[(i >> 5) + 1] += v;
                    else
                        a[i >> 5] += v;
                }
                // 32 distances at a time, from the nearest on; a lane adds up a bucket's.
                float *run = small + 256 + 32 * warp;
#pragma unroll
                for (int r = 2; r >= 0; --r) {
                    const int base = p_lo + quarter * 32 - key0 - 32 * r;
                    __syncwarp();
                    run[lane] = a[r];
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int b = lane + 32 * k;
                        if (b < p.bias.num_buckets) {
                            const int lo = max(p.bias.first[b] - base, 0), hi = min(p.bias.first[b + 1] - base, 32);
                            for (int x = lo; x < hi; ++x) by_bucket[k] += run[x];
                        }
                    }
                }
            }
        }
        if (wait_warp(bar(B_DONE), 0, c.abort_flag, p.err, kTimeoutNs)) {
            tc_fence_after();
            const bool v8 = aligned32(p.dq, p.dq_stride);
            __nv_bfloat16 *dst = dq + static_cast<int64_t>(row) * p.dq_stride + wg * (HD / 2);
#pragma unroll 1
            for (int cc = 0; cc < HD / 64; ++cc)
                store_chunk(c.tmem + t_lane + kDq + wg * (HD / 2) + cc * 32, p.scale, dst + cc * 32, valid, v8);
            // What is left to add up goes to K's first stage, which no copy or product uses any more:
            // the last bucket's half sums of the rows, the warps' buckets.
            if constexpr (BIAS) {
                float *sums = reinterpret_cast<float *>(c.sb + L::OFF_A);
                sums[256 * wg + row] = d_far;
                sums[256 * wg + 128 + row] = w_far;
#pragma unroll
                for (int k = 0; k < 4; ++k) sums[512 + 128 * warp + lane + 32 * k] = by_bucket[k];
            }
            if (n_pre == n) small[128 * wg + row] = d_sum;
        }
    }
    teardown(c);
    if (*c.abort_flag) return;
    // (The half sums of D are in `small` either way.)
    float far_sum = 0.f;
    const float *sums = reinterpret_cast<const float *>(c.sb + L::OFF_A);
    if (threadIdx.x < rows) {
        const float d = small[threadIdx.x] + small[128 + threadIdx.x];
        p.delta[stat_row + threadIdx.x] = d;
        if constexpr (BIAS)
            far_sum = sums[threadIdx.x] + sums[256 + threadIdx.x] - d * (sums[128 + threadIdx.x] + sums[384 + threadIdx.x]);
    }
    if constexpr (BIAS) {
        __syncthreads();
        far_sum = warp_sum(far_sum);
        if (lane == 0) small[warp] = far_sum;  // (warps 4 on: 0)
        __syncthreads();
        const int b = threadIdx.x;
        if (b < p.bias.num_buckets) {
            float t = b == p.bias.num_buckets - 1 ? (small[0] + small[1]) + (small[2] + small[3]) : 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) t += sums[512 + 128 * w + b];
            p.partial[((static_cast<int64_t>(s.q_start / BM) + seq + qt) * p.num_heads + h) * p.bias.num_buckets + b] = t;
        }
    }
}

// --------------------------------------------------------------------- dK, dV ---
// Tensor memory: S^T (then P^T) at 0, dP^T (then dS^T) at 128, dV at 256, dK at 384.  While the
// element-wise warps form P^T, the tensor cores run dK of the tile before and dP^T; while they form
// dS^T, dV and the next tile's S^T:
//     dP(i), dV(i), S(i + 1), dK(i).
template <int HD, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) grad_kv_kernel(const __grid_constant__ GradParams p) {
    using L = LayoutKv<HD>;
    constexpr uint32_t kS = 0, kDp = 128, kDv = 256, kDk = 384;
    const int kvh = blockIdx.x % p.num_kv_heads;
    const int rest = blockIdx.x / p.num_kv_heads;
    const int seq = rest % p.num_seqs;
    const int kt = rest / p.num_seqs;  // the first keys are seen by the most rows
    const Seq s = load_seq(p, seq, false);
    const int k_lo = kt * BM;
    if (!s.ok || k_lo >= s.sk) return;
    const int rows = min(BM, s.sk - k_lo);
    const int off = s.sk - s.sq;  // position of the first query
    const int r_first = max(0, k_lo - off);
    int r_end = s.sq;
    if (p.window > 0) r_end = static_cast<int>(min(static_cast<int64_t>(r_end), static_cast<int64_t>(k_lo) + rows - 1 + p.window - off));
    const int nq = r_end > r_first ? (r_end - r_first + BN - 1) / BN : 0;
    const int n = nq * p.group;
    __nv_bfloat16 *dk = p.dk + (static_cast<int64_t>(s.k_start) + k_lo) * p.dk_stride + kvh * HD;
    __nv_bfloat16 *dv = p.dv + (static_cast<int64_t>(s.k_start) + k_lo) * p.dv_stride + kvh * HD;
    if (n == 0) {  // no row sees these keys
        zero_rows<HD>(dk, p.dk_stride, rows);
        zero_rows<HD>(dv, p.dv_stride, rows);
        return;
    }
    const Cta c = setup<L>();
    auto bar = [&](int i) -> uint32_t { return c.base + L::OFF_BAR + 8u * static_cast<uint32_t>(i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sK = c.base + L::OFF_RES, sV = sK + L::TILE;
    auto sQ = [&](int st) -> uint32_t { return c.base + L::OFF_A + st * L::TILE; };
    auto sDo = [&](int st) -> uint32_t { return c.base + L::OFF_B + st * L::TILE; };
    // Per stage: -lse2, -D and (BIAS) the last bucket's bias - lse2 of the tile's queries.
    auto stat = [&](int st) -> float * { return reinterpret_cast<float *>(c.sb + L::OFF_SMALL) + st * 384; };
    const int last = p.bias.last();

    if (warp == kWarpLoad) {
        if (lane < 4) prefetch_tmap(lane == 0 ? p.tmap_q : lane == 1 ? p.tmap_do : lane == 2 ? p.tmap_k : p.tmap_v);
        if (lane == 0) mbar_arrive_expect_tx(bar(B_RES), 2 * L::TILE);
        __syncwarp();
        load_tile<HD>(p.tmap_k, sK, kvh, s.k_start, k_lo, s.sk, bar(B_RES));
        load_tile<HD>(p.tmap_v, sV, kvh, s.k_start, k_lo, s.sk, bar(B_RES));
        uint32_t lands = 0;
        int g = 0, t = 0;
        for (int i = 0; i < n; ++i) {
            const int st = i & 1;
            const int r = r_first + t * BN, head = kvh * p.group + g;
            // (dout's stage is free first: dV comes before dK.)
            if (i >= 2 && !wait_warp(bar(B_BEMPTY + st), ((i >> 1) - 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
            if (!load_stage<HD>(p.tmap_do, sDo(st), head, s.q_start, r, s.sq, bar(B_BFULL + st), bar(B_LAND), lands, c.abort_flag, p.err, [] {})) break;
            if (i >= 2 && !wait_warp(bar(B_AEMPTY + st), ((i >> 1) - 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
            auto stats = [&] {
                float far = 0.f;
                if constexpr (BIAS) far = __ldg(bias_row_of(p.bias_table, head, last) + last);
                const int64_t at = static_cast<int64_t>(head) * p.total_q + s.q_start + r;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int x = lane + 32 * e;
                    const bool in = r + x < s.sq;
                    const float l2 = in ? p.lse2[at + x] : INFINITY;
                    stat(st)[x] = -l2;
                    stat(st)[128 + x] = in ? -p.delta[at + x] : 0.f;
                    if constexpr (BIAS) stat(st)[256 + x] = far - l2;
                }
            };
            if (!load_stage<HD>(p.tmap_q, sQ(st), head, s.q_start, r, s.sq, bar(B_AFULL + st), bar(B_LAND), lands, c.abort_flag, p.err, stats)) break;
            if (++t == nq) {
                t = 0;
                ++g;
            }
        }
    } else if (warp == kWarpMma) {
        if (lane == 0) {
            auto wait = [&](int b, uint32_t parity) { return wait1(bar(b), parity, c.abort_flag, p.err, kTimeoutNs); };
            bool ok = wait(B_RES, 0) && wait(B_AFULL, 0);
            if (ok) {
                tc_fence_after();
                issue_abt<HD>(c.tmem + kS, sK, sQ(0));
                mma_commit(bar(B_SFULL));
            }
            for (int i = 0; ok && i < n; ++i) {
                const int st = i & 1;
                ok = wait(B_BFULL + st, (i >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                issue_abt<HD>(c.tmem + kDp, sV, sDo(st));
                mma_commit(bar(B_DPFULL));
                ok = wait(B_PFULL, i & 1);
                if (!ok) break;
                tc_fence_after();
                issue_ab<HD>(c.tmem + kDv, c.tmem + kS, sDo(st), i == 0);
                mma_commit(bar(B_BEMPTY + st));
                if (i + 1 < n) {
                    const int sn = (i + 1) & 1;
                    ok = wait(B_AFULL + sn, ((i + 1) >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    issue_abt<HD>(c.tmem + kS, sK, sQ(sn));
                    mma_commit(bar(B_SFULL));
                }
                ok = wait(B_DSFULL, i & 1);
                if (!ok) break;
                tc_fence_after();
                issue_ab<HD>(c.tmem + kDk, c.tmem + kDp, sQ(st), i == 0);
                mma_commit(bar(B_AEMPTY + st));
            }
            if (ok) mma_commit(bar(B_DONE));
        }
    } else {
        const int wg = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
        const float sl2 = p.scale_log2;
        const int key = k_lo + row;
        const uint32_t sc = c.tmem + t_lane + kS + 64u * wg, dp = c.tmem + t_lane + kDp + 64u * wg;
        int g = 0, t = 0;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int st = i & 1;
            const int pos0 = off + r_first + t * BN + 64 * wg;  // position of this warpgroup's first query
            if (!wait_warp(bar(B_AFULL + st), (i >> 1) & 1, c.abort_flag, p.err, kTimeoutNs) ||
                !wait_warp(bar(B_SFULL), i & 1, c.abort_flag, p.err, kTimeoutNs)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float w[2][32];
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) tmem_ld_32x32b_x32(sc + 32u * cc, w[cc]);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) tmem_wait_ld_regs(w[cc]);
            const int d0 = pos0 - key;  // distance from the first query
            bool near = false;
            // (lane 31 has the nearest key)
            if constexpr (BIAS) near = __shfl_sync(0xffffffffu, d0, 31) < last && __shfl_sync(0xffffffffu, d0, 0) + 63 >= 0;
            if (near) {
                const float *bt = bias_row_of(p.bias_table, kvh * p.group + g, last) + d0;
                const float4 *nl = reinterpret_cast<const float4 *>(stat(st) + 64 * wg);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float4 l = nl[x];
                    float *v = &w[x >> 3][4 * (x & 7)];
                    v[0] = fmaf(v[0], sl2, __ldg(bt + 4 * x)) + l.x;
                    v[1] = fmaf(v[1], sl2, __ldg(bt + 4 * x + 1)) + l.y;
                    v[2] = fmaf(v[2], sl2, __ldg(bt + 4 * x + 2)) + l.z;
                    v[3] = fmaf(v[3], sl2, __ldg(bt + 4 * x + 3)) + l.w;
                }
            } else {
                const ulonglong2 *nl = reinterpret_cast<const ulonglong2 *>(stat(st) + (BIAS ? 256 : 0) + 64 * wg);
                const uint64_t sl2x2 = f2_pack(sl2, sl2);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const ulonglong2 l = nl[x];
                    float *v = &w[x >> 3][4 * (x & 7)];
                    f2_unpack(f2_fma(f2_pack(v[0], v[1]), sl2x2, l.x), v[0], v[1]);
                    f2_unpack(f2_fma(f2_pack(v[2], v[3]), sl2x2, l.y), v[2], v[3]);
                }
            }
            if (d0 < 0) {
#pragma unroll
                for (int x = 0; x < 64; ++x)
                    if (x < -d0) w[x >> 5][x & 31] = -INFINITY;
            }
            if (p.window > 0 && d0 + 63 >= p.window) {
                const int end = p.window - d0;  // queries from here on are too far
#pragma unroll
                for (int x = 0; x < 64; ++x)
                    if (x >= end) w[x >> 5][x & 31] = -INFINITY;
            }
            uint32_t pk[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                float &a = w[x >> 4][2 * (x & 15)], &b = w[x >> 4][2 * (x & 15) + 1];
                a = ex2_approx(a);
                b = ex2_approx(b);
                pk[x] = pack_bf16x2(a, b);
            }
            tmem_st_32x32b_x32_u(sc, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_PFULL));
            if (!wait_warp(bar(B_DPFULL), i & 1, c.abort_flag, p.err, kTimeoutNs)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const ulonglong2 *dl = reinterpret_cast<const ulonglong2 *>(stat(st) + 128 + 64 * wg);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                float d[32];
                tmem_ld_32x32b_x32(dp + 32u * cc, d);
                tmem_wait_ld_regs(d);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const ulonglong2 l = dl[8 * cc + x];
                    float *v = &d[4 * x];
                    const float *pw = &w[cc][4 * x];
                    f2_unpack(f2_mul(f2_pack(pw[0], pw[1]), f2_add(f2_pack(v[0], v[1]), l.x)), v[0], v[1]);
                    f2_unpack(f2_mul(f2_pack(pw[2], pw[3]), f2_add(f2_pack(v[2], v[3]), l.y)), v[2], v[3]);
                    pk[16 * cc + 2 * x] = pack_bf16x2(v[0], v[1]);
                    pk[16 * cc + 2 * x + 1] = pack_bf16x2(v[2], v[3]);
                }
            }
            tmem_st_32x32b_x32_u(dp, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DSFULL));
            if (++t == nq) {
                t = 0;
                ++g;
            }
        }
        if (ok && wait_warp(bar(B_DONE), 0, c.abort_flag, p.err, kTimeoutNs)) {
            tc_fence_after();
            const int64_t stride = wg ? p.dk_stride : p.dv_stride;
            __nv_bfloat16 *dst = (wg ? dk : dv) + static_cast<int64_t>(row) * stride;
            const bool v8 = aligned32(wg ? p.dk : p.dv, stride);
#pragma unroll 1
            for (int cc = 0; cc < HD / 32; ++cc)
                store_chunk(c.tmem + t_lane + (wg ? kDk : kDv) + cc * 32, wg ? p.scale : 1.f, dst + cc * 32, row < rows, v8);
        }
    }
    teardown(c);
}

// ---------------------------------------------------------------------- dbias ---
// Sums the query tiles' partial sums in their order, a block a head.
__global__ void __launch_bounds__(1024)
    grad_bias_kernel(float *__restrict__ dbias, const float *__restrict__ partial, int slots, int num_heads, int num_buckets) {
    __shared__ float s[8][128];
    const int h = blockIdx.x, b = threadIdx.x & 127, part = threadIdx.x >> 7;
    float t = 0.f;
    if (b < num_buckets)
        for (int i = part; i < slots; i += 8) t += partial[(static_cast<int64_t>(i) * num_heads + h) * num_buckets + b];
    s[part][b] = t;
    __syncthreads();
    if (part == 0 && b < num_buckets) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[i][b];
        dbias[b * num_heads + h] = t;
    }
}

// ------------------------------------------------------------------ host side ---
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Query tiles of all sequences: tile t of sequence i has place cu_seqlens_q[i] / 128 + i + t.
int64_t tile_slots(int total_q, int num_seqs) { return static_cast<int64_t>(total_q) / BM + num_seqs + 1; }

template <class Kernel>
cudaError_t launch_tiles(Kernel kern, uint32_t smem, std::atomic<uint64_t> &set, int64_t blocks, const GradParams &p,
                         cudaStream_t stream) {
    if (blocks <= 0) return cudaSuccess;
    const cudaError_t e = smem_limit_once(kern, static_cast<int>(smem), set);
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int HD, bool BIAS>
cudaError_t launch_backward_d(GradParams &p, const PackedGradArgs &g, cudaStream_t stream) {
    const PackedArgs &a = g.fwd;
    const int64_t rows = static_cast<int64_t>(a.num_heads) * HD;
    // (Without queries, or keys, nothing is loaded, but a tensor map has a row and an address.)
    auto rows_map = [](CUtensorMap *map, const void *base, const void *spare, int heads, int total, int64_t stride) {
        for (int i = 0; i < 2; ++i)
            if (!encode_3d(map + i, total > 0 ? base : spare, HD, heads, total > 0 ? total : 1, HD * 2, stride * 2, 64, 1, i ? 16 : 128))
                return false;
        return true;
    };
    if (!rows_map(p.tmap_q, a.q, a.k, a.num_heads, a.total_q, a.q_stride) ||
        !rows_map(p.tmap_do, g.dout, a.k, a.num_heads, a.total_q, rows) ||
        !rows_map(p.tmap_k, a.k, a.q, a.num_kv_heads, a.total_k, a.k_stride) ||
        !rows_map(p.tmap_v, a.v, a.q, a.num_kv_heads, a.total_k, a.v_stride))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (a.total_q > 0) {
        const dim3 grid((a.total_q + 7) / 8, (a.num_heads + 7) / 8);
        grad_stat_kernel<HD><<<grid, 256, 0, stream>>>(static_cast<const uint4 *>(g.out), static_cast<const uint4 *>(g.dout), g.lse,
                                                       const_cast<float *>(p.lse2), p.delta, a.total_q, a.num_heads);
        e = cudaGetLastError();
    }
    static std::atomic<uint64_t> set[2];
    const int64_t q_blocks = static_cast<int64_t>(p.q_tiles) * a.num_seqs * a.num_heads;
    const int64_t k_blocks = (static_cast<int64_t>(a.max_seqlen_k) + BM - 1) / BM * a.num_seqs * a.num_kv_heads;
    const int slots = static_cast<int>(tile_slots(a.total_q, a.num_seqs));
    if (BIAS && e == cudaSuccess)  // (places without a tile)
        e = cudaMemsetAsync(p.partial, 0, static_cast<size_t>(slots) * a.num_heads * a.bias.num_buckets * sizeof(float), stream);
    if (e == cudaSuccess) e = launch_tiles(grad_q_kernel<HD, BIAS>, LayoutQ<HD>::SMEM, set[0], q_blocks, p, stream);
    if (e == cudaSuccess) e = launch_tiles(grad_kv_kernel<HD, BIAS>, LayoutKv<HD>::SMEM, set[1], k_blocks, p, stream);
    if constexpr (BIAS) {
        if (e != cudaSuccess) return e;
        grad_bias_kernel<<<a.num_heads, 1024, 0, stream>>>(g.dbias, p.partial, slots, a.num_heads, a.bias.num_buckets);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

bool packed_grad_workspace(int total_q, int num_seqs, int num_heads, int num_buckets, size_t *bytes) {
    const int64_t slots = tile_slots(total_q, num_seqs);
    if (slots * num_heads > INT_MAX) return false;
    *bytes = 2 * up256(static_cast<size_t>(total_q) * num_heads * sizeof(float)) +
             up256(static_cast<size_t>(slots) * num_heads * num_buckets * sizeof(float));
    return true;
}

cudaError_t launch_packed_attn_backward(const PackedGradArgs &g, cudaStream_t stream) {
    const PackedArgs &a = g.fwd;
    GradParams p;
    memset(&p, 0, sizeof p);
    p.cu_q = a.cu_seqlens_q;
    p.cu_k = a.cu_seqlens_k;
    p.dq = static_cast<__nv_bfloat16 *>(g.dq);
    p.dk = static_cast<__nv_bfloat16 *>(g.dk);
    p.dv = static_cast<__nv_bfloat16 *>(g.dv);
    p.dq_stride = g.dq_stride;
    p.dk_stride = g.dk_stride;
    p.dv_stride = g.dv_stride;
    uint8_t *ws = static_cast<uint8_t *>(g.workspace);
    const size_t stat = up256(static_cast<size_t>(a.total_q) * a.num_heads * sizeof(float));
    p.lse2 = reinterpret_cast<const float *>(ws);
    p.delta = reinterpret_cast<float *>(ws + stat);
    p.partial = reinterpret_cast<float *>(ws + 2 * stat);
    p.bias_table = a.bias_table;
    p.num_seqs = a.num_seqs;
    p.total_q = a.total_q;
    p.total_k = a.total_k;
    p.max_q = a.max_seqlen_q;
    p.max_k = a.max_seqlen_k;
    p.q_tiles = static_cast<int>((static_cast<int64_t>(a.max_seqlen_q) + BM - 1) / BM);
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.group = a.num_heads / a.num_kv_heads;
    p.window = a.sliding_window;
    p.scale = a.scale;
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    p.bias = a.bias;
    const bool bias = a.bias_table != nullptr;
    switch (a.head_dim) {
        case 64: return bias ? launch_backward_d<64, true>(p, g, stream) : launch_backward_d<64, false>(p, g, stream);
        case 128: return bias ? launch_backward_d<128, true>(p, g, stream) : launch_backward_d<128, false>(p, g, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
