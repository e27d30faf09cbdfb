// attn_backward.cu - gradient of packed variable-length attention on the sm_103a tensor cores
// (tcgen05 + TMEM).
//
// With s_ij = scale q_i k_j + bias(p_i - j), P_ij = e^(s_ij - lse_i) over the keys j that row i sees,
// out = P V and dout given:
//     dP = dout V^T,   D_i = sum_j P_ij dP_ij,   dS = P (dP - D),
//     dV = P^T dout,   dQ = scale dS K,   dK = scale dS^T Q,   dbias_b = sum of dS over bucket b.
// D_i also equals dout_i out_i, but out is bf16 there: good enough inside dQ, whose terms are rounded
// to bf16 anyway, unless a row's dS nearly cancel, as they do where few keys have the weight; and not
// for sums of dS.  So the dQ kernel starts from dout_i out_i, visits the tiles that need the sum itself once
// for D and once with it, and leaves D in fp32 for dK.  What dout_i out_i was off by is known at an item's
// end; where that is more than the rounding of dS may be, for any row, the item is done again with D.
//
// Two kernels share the work, each with its accumulators in tensor memory and no atomics, so equal
// calls give equal bits:
//  * grad_q_kernel: 128 queries of one head against their keys in turn (3 products a tile).  dbias: the
//    tiles whose distances all belong to the last bucket add sum_j P dP - D sum_j P to it; the others,
//    the nearest ones, come last, and their dS, with the exact D, are summed along diagonals into
//    buckets;
//  * grad_kv_kernel: 128 keys of one kv head against the queries of every head that shares it
//    (4 products a tile), so the sum over the heads happens in the accumulator.
// The products count 7 for the 5 of the formula (S and dP are formed twice); dQ added up across
// the CTAs of one pass over the keys would need atomics, whose order changes the result.
//
// Persistent CTAs, one an SM, take (tile, head) items from a list sorted by the number of steps,
// dealt in snake order: a CTA's start, about 6600 cycles to its first product, is paid once, and an
// item's loads run during the end of the one before.
//
// Roles in a CTA: warps 0-7 are two warpgroups of element-wise work, each on 64 of a tile's 128
// columns (a warp on the 32 lanes of tensor memory that it can reach); warp 8 loads tiles by TMA, warp 9
// (in dQ with warp 10) issues the products.  P and dS go back to tensor memory as bf16, over the fp32
// tile they came from, and are the first operand of the next product from there.
//
// Measured (packed sequences, 32/8 heads of 128; the products of each kernel over its time):
//  * two of 6000-8192 tokens, no bias: dQ 717 us (1.57 PFLOP/s of three products, 0.81 of the bf16
//    peak; 657 us without the sums of |dS| that tell which rows are done again, 1380-1420 where nearly all
//    are, with queries three or four times as large), dK/dV 900 us (1.67);
//  * sixteen of 128-2048 tokens, 32 buckets to 128: dQ 316 us (0.75; 295 and 590), dK/dV 281 us (1.14).  A block of
//    dQ takes 216 steps, 58 of them near tiles, in 30 items of which the last step's chain (logits, D,
//    dS, diagonals, product, rows out) has nothing beside it;
//  * 128 of 128 tokens, where an item is one step: dQ 104 us without a bias (the bytes alone take 69),
//    130 with one, dK/dV 77 and 79 (59).
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
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpMma2 = 10;
constexpr int kThreads = 384;  // (whole warpgroups: the last warp has no work)
constexpr uint32_t kTmemCols = 512;
// Rows of fewer keys get their D from the sum over the keys at once also for dQ: few keys share their weight, so
// that dout . out would mostly have to be done again, and they have two tiles at most.
constexpr int kFewKeys = 128;
// A row is done again with D if dout . out, off by x, moves its dS by more in all (x times the weights of
// the tiles that took it) than half a step of bf16 of each: dout . out is off by about 2^-9 of the root of its terms'
// squares, so that a weight spread over ten keys or more never is.  Items (128 rows of a head) done again with 2048 keys: none
// with logits of standard deviation 1, 12 % with 2, nearly all from 3 on, which take twice the products then.
constexpr float kMoved = 0.00390625f;
// Rows whose lse lies below see nothing but keys with biases that stand for hiding them (-1e9, say).  P = e^(s - lse) is off by
// a factor of up to e^(2^-22 |lse|), 1.3 here and anything from 0 to infinity at -1e9: they have no gradient, as rows without keys.
constexpr float kNoDigits = -1.0e6f;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per wait

// 128 queries of a sequence.
struct alignas(16) QTile {
    int row;      // first row of q
    int left;     // rows from there to the sequence's end (1 ..)
    int pos;      // position of the first row (negative: it sees no key)
    int k_start;  // first row of k
    int sk;       // keys
    int n;        // tiles of 128 keys that some row sees
    int id;       // place among all query tiles in the sequences' order
    int pad;
};
// 128 keys of a sequence, or a part of their steps: one for each head of the kv head and each tile of 128
// queries that sees some of the keys.
struct alignas(16) KTile {
    int row;      // first row of k
    int left;     // rows from there to the sequence's end (1 ..)
    int key;      // position of the first key
    int off;      // position of the first query
    int q_start;  // first row of q
    int sq;       // queries
    int n;        // tiles of 128 queries
    int from, to;  // steps of this part, of n times the heads of a kv head
    int part, parts;
    int slot;     // (parts > 1) of the first part of kv head 0
};

struct GradParams {
    // Boxes of 64 dims of one head: [0] of 128 rows, [1] of 16 rows.
    CUtensorMap tmap_q[2];
    CUtensorMap tmap_do[2];
    CUtensorMap tmap_k[2];
    CUtensorMap tmap_v[2];
    __nv_bfloat16 *dq;
    __nv_bfloat16 *dk;
    __nv_bfloat16 *dv;
    int64_t dq_stride, dk_stride, dv_stride;
    const float *lse2;  // [num_heads, total_q]: lse in base 2, +inf for a row without keys (or with an lse below kNoDigits)
    float *delta;       // [num_heads, total_q]: D
    const float *bias_table;
    float *partial;     // [query tiles, num_heads, 8 warps, num_buckets]
    const int *counts;  // [2]: query tiles, key tiles
    const QTile *q_list;
    const KTile *k_list;
    float *split;       // [slots][dV, dK][HD / 4][128 rows][4]: sums of key tiles whose steps are split
    int *arrived;       // [slots][8 warps]
    uint8_t *again;     // [query tiles, num_heads][4 warps]: whether a warp's rows are done again with D
    int total_q, total_k;
    int num_heads, num_kv_heads, group;
    int window;
    float scale, scale_log2;
    unsigned *err;
    RelativeBias bias;
};

// First key tile of a query tile, and first query of a key tile.
__device__ __forceinline__ int first_key(int pos, int window) { return window > 0 ? max(0, pos - window + 1) : 0; }
__device__ __forceinline__ int first_query(const KTile &t) { return max(0, t.key - t.off); }

// Item k of a CTA: (list entry, head), in snake order over the CTAs.  False: no more.
__device__ __forceinline__ bool item_of(int k, int count, int heads, int &entry, int &head) {
    const int64_t g = gridDim.x;
    const int64_t v = k * g + ((k & 1) ? g - 1 - blockIdx.x : blockIdx.x);
    if (v >= static_cast<int64_t>(count) * heads) return false;
    entry = static_cast<int>(v / heads);
    head = static_cast<int>(v - static_cast<int64_t>(entry) * heads);
    return true;
}
// The first item from k on that is done again (by a whole warp); beyond all items: none.
__device__ __forceinline__ int next_again(int k, int count, int heads, const uint8_t *again) {
    for (;; k += 32) {
        int entry, head;
        const bool have = item_of(k + (threadIdx.x & 31), count, heads, entry, head);
        const uint32_t f =
            have ? __ldcg(reinterpret_cast<const unsigned *>(again) + static_cast<int64_t>(entry) * heads + head) : 0u;
        const uint32_t m = __ballot_sync(0xffffffffu, f != 0u);
        if (m != 0u) return k + __ffs(m) - 1;
        if (!__all_sync(0xffffffffu, have)) return INT_MAX;
    }
}
template <class Tile>
__device__ __forceinline__ Tile load_entry(const Tile *list, int i) {
    static_assert(sizeof(Tile) % 16 == 0, "entries are read as 16-byte vectors");
    Tile t;
    int *d = reinterpret_cast<int *>(&t);
#pragma unroll
    for (int x = 0; x < static_cast<int>(sizeof(Tile) / 16); ++x) {
        const int4 a = __ldg(reinterpret_cast<const int4 *>(list + i) + x);
        d[4 * x] = a.x, d[4 * x + 1] = a.y, d[4 * x + 2] = a.z, d[4 * x + 3] = a.w;
    }
    return t;
}

// Shared memory: two resident tiles (Q and dout, or K and V; with heads of 64 there is room for the next
// item's, whose loads then hide behind this one's work), rings of the tiles that pass by (K and V, or Q
// and dout), small arrays, barriers.  K outlives V by the time from dP to dQ, so it has
// three stages there.  With a bias and heads of 128, V's second stage gives nothing (16 sequences of
// 128-2048 tokens, 32/8 heads: the same time with and without it), and its place holds the bias of two
// items' heads.
template <int HD, int STAGES_A, int STAGES_B, uint32_t SMALL_BYTES>
struct Layout {
    static constexpr int NHALF = HD / 64;
    static constexpr uint32_t TILE = NHALF * HALF;
    static constexpr int NR = HD == 64 ? 2 : 1, NA = STAGES_A, NB = STAGES_B;
    static constexpr uint32_t OFF_RES = 0;
    static constexpr uint32_t OFF_A = 2 * NR * TILE;     // Q (dK, dV) or K (dQ)
    static constexpr uint32_t OFF_B = OFF_A + NA * TILE;  // dout (dK, dV) or V (dQ)
    static constexpr uint32_t OFF_SMALL = OFF_B + NB * TILE;
    static constexpr uint32_t OFF_BAR = OFF_SMALL + SMALL_BYTES;
    static constexpr uint32_t OFF_MISC = OFF_BAR + 240;
    static constexpr uint32_t BYTES = OFF_MISC + 16;
    // At least 116 KB so a single CTA owns an SM (and all of its TMEM).
    static constexpr uint32_t SMEM = (BYTES > 118784u ? BYTES : 118784u);
    static_assert(SMEM <= 232448u, "at most 227 KB of shared memory per CTA");
};

// An item's bias (dK, dV: of its kv head's heads) in shared memory; a longer one is read from global memory.
constexpr uint32_t kTableBytesQ = 13312, kTableBytes = 15360;
// What is kept of a head's row: distances -kNearPad .. last + 127.
constexpr int kNearPad = 256;
__host__ __device__ constexpr int near_entries(int last) { return (last + kNearPad + 128 + 3) & ~3; }
// dQ's small arrays, as floats: two items' halves of D, and of the second half of the columns (in bf16, rounded to the safe side) the
// sums of |dS|; with a bias those of P, the buckets' first distances and each warp's sums along diagonals.
constexpr int kAbsAt = 512, kWeightAt = kAbsAt + 128, kFirstAt = kWeightAt + 128, kDiagAt = kFirstAt + 132;
constexpr uint32_t kSmallQ = 4u * kWeightAt, kSmallQBias = 4u * (kDiagAt + 8 * 96);
static_assert(kSmallQBias % 16 == 0, "the bias behind it comes by bulk copies");
template <int HD, bool BIAS>
using LayoutQ = Layout<HD, 3, BIAS && HD == 128 ? 1 : 2, BIAS ? kSmallQBias + 2 * kTableBytesQ : kSmallQ>;
constexpr uint32_t kSmallKv = 2u * 3 * 512;
template <int HD, bool BIAS>
using LayoutKv = Layout<HD, 2, 2, kSmallKv + (BIAS ? 2 * kTableBytes : 0u)>;

enum : int {
    B_RES = 0,        // [2] resident tiles loaded (the second one's at 28)
    B_RESEMPTY = 20,  // [2] resident tiles read (the second one's at 29)
    B_ACCFREE = 21,   // accumulators stored (8 warps)
    B_AFULL = 1,    // [3] tile of ring A ready (dK, dV: of both rings, and a second arrival for the rows' statistics)
    B_AEMPTY = 4,   // [3] read
    B_BFULL = 7,    // [2] ring B
    B_BEMPTY = 9,   // [2]
    B_LAND = 11,    // copies of a tile that the loading warp edits
    B_SFULL = 12,   // logits of a tile ready
    B_PFULL = 13,   // logits read (dQ), or P in tensor memory (dK, dV) (8 warps)
    B_DPFULL = 14,  // [2] dP ready
    B_DSFULL = 16,  // [2] dS in tensor memory (8 warps)
    B_DONE = 18,    // all products done
    B_SUMS = 19,    // both halves of the rows' D written (8 warps)
    B_DQDONE = 22,    // [2] dQ's product of a step done
    B_TABFULL = 24,   // [2] an item's bias in shared memory
    B_TABFREE = 26,   // [2] read (8 warps)
    NBARS = 30
};
__device__ __forceinline__ int res_full(uint32_t slot) { return slot ? 28 : B_RES; }
__device__ __forceinline__ int res_empty(uint32_t slot) { return slot ? 29 : B_RESEMPTY; }

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
// By the element-wise warps.
template <int HD>
__device__ __forceinline__ void zero_rows(__nv_bfloat16 *dst, int64_t stride, int rows) {
    for (int i = threadIdx.x; i < rows * (HD / 8); i += 256)
        *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(i / (HD / 8)) * stride + i % (HD / 8) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
}

// A warp's 32 x 64 block of a tile as the element-wise warps hold it: thread t has the rows t / 4 + 8 a
// (a = 0 .. 3) and of each the columns 8 b + 2 (t % 4) + e (b = 0 .. 7, e = 0, 1), from two loads of 16 lanes.
// Row - column is then the same for all (a, b) with the same a - b, 11 pairs of distances for 64 elements:
// a bias costs a thread 22 reads, masks are 22 comparisons, and sums along diagonals begin with additions in
// registers.  (A thread a row needs 64 reads, comparisons and shuffles: dQ of 16 sequences of 128-2048 tokens,
// 32/8 heads of 128 took 375 us that way, 318 this way; without a bias of two documents of 6000-8192 tokens
// 648 against 664.  Both before what followed.)
__device__ __forceinline__ int pair_at(int a, int b) { return 4 * b + 2 * (a & 1); }
__device__ __forceinline__ uint64_t block_pair(const float (&w)[2][32], int a, int b) {
    return f2_pack(w[a >> 1][pair_at(a, b)], w[a >> 1][pair_at(a, b) + 1]);
}
__device__ __forceinline__ void set_pair(float (&w)[2][32], int a, int b, uint64_t x) {
    f2_unpack(x, w[a >> 1][pair_at(a, b)], w[a >> 1][pair_at(a, b) + 1]);
}
__device__ __forceinline__ void load_block(uint32_t taddr, float (&w)[2][32]) {
    tmem_ld_16x256b_x8(taddr, w[0]);
    tmem_ld_16x256b_x8(taddr + (16u << 16), w[1]);
    tmem_wait_ld_regs(w[0]);
    tmem_wait_ld_regs(w[1]);
}
__device__ __forceinline__ float pair_sum(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    return a + b;
}

// Shared set-up of both kernels.
struct Cta {
    uint32_t base;
    uint8_t *sb;
    uint32_t tmem;
    volatile int *abort_flag;
    volatile int *again;  // (dQ) some item is done again
};
template <class L>
__device__ __forceinline__ Cta setup(int full_arrivals) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];  // (swizzled tiles start on 1024 bytes)
    Cta c;
    c.base = smem_u32(smem_raw);
    c.sb = smem_raw;
    c.abort_flag = reinterpret_cast<volatile int *>(c.sb + L::OFF_MISC + 4);
    c.again = reinterpret_cast<volatile int *>(c.sb + L::OFF_MISC + 8);
    auto bar = [&](int i) -> uint32_t { return c.base + L::OFF_BAR + 8u * static_cast<uint32_t>(i); };
    if (threadIdx.x == 0) {
        mbar_init(bar(B_ACCFREE), 8);
        for (int s = 0; s < 3; ++s) {
            mbar_init(bar(B_AFULL + s), full_arrivals);
            mbar_init(bar(B_AEMPTY + s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(res_full(s)), 1);
            mbar_init(bar(res_empty(s)), 1);
            mbar_init(bar(B_BFULL + s), full_arrivals);
            mbar_init(bar(B_BEMPTY + s), 1);
            mbar_init(bar(B_DPFULL + s), 1);
            mbar_init(bar(B_DSFULL + s), 8);
            mbar_init(bar(B_DQDONE + s), 1);
            mbar_init(bar(B_TABFULL + s), 1);
            mbar_init(bar(B_TABFREE + s), 8);
        }
        mbar_init(bar(B_LAND), 1);
        mbar_init(bar(B_SFULL), 1);
        mbar_init(bar(B_PFULL), 8);
        mbar_init(bar(B_DONE), 1);
        mbar_init(bar(B_SUMS), 8);
        *c.abort_flag = 0;
        *c.again = 0;
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

// ------------------------------------------------- lists and rows' statistics ---
// The tiles of all sequences, sorted by their number of steps (the longest first), by one block.  A
// warp takes 32 sequences at a time, a lane a tile; the order of equal tiles is left to chance (no
// result depends on it).  Bad sequences are flagged and have no tiles; offsets that go back and forth can
// give sequences that share rows more tiles than the lists hold, and then none has any.
struct PlanParams {
    const int32_t *cu_q;
    const int32_t *cu_k;
    int num_seqs, total_q, total_k, max_q, max_k, window;
    int most[2];  // tiles that the lists have room for (the key tiles' also for the parts of those that are split)
    int num_kv_heads, group;
    int slots;    // places for the sums of split key tiles
    int *arrived;
    int *counts;
    QTile *q_list;
    KTile *k_list;
    unsigned *err;
};
constexpr int kPlanBins = 1024;  // longer tiles share the last bin
// Key tiles of more steps than an SM's share and 8 more are split: few kv heads with many queries each have
// few long items.  dK/dV with and without, us: one sequence of 2048, 32/8 heads of 128 71 and 97, 16/1 57 and
// 348; of 4096, 32/4 heads of 64 184 and 301, 8/2 of 128 65 and 177; of 16384, 8/1 of 128 820 and 1367; of 3000
// and 1100, 16/2 of 64 60 and 219.  Where an SM's share is nearly a tile's steps the parts cost more than they even
// out: 4096, 32/8 of 128 204 and 181.  Parts leave their sums in fp32; the last one to arrive, warp by warp,
// adds them up in the parts' order.  A part costs about five steps, for its keys and its sums.  So many
// slots suffice: a split tile has fewer parts than twice its steps over an SM's share.
constexpr int kMinSteps = 8, kMaxSlots = 2 * kPlanSms + 1;

// emit(chunk of sequences, tile of the chunk, tile of the sequence, the sequence)
template <class Emit, class Chunk>
__device__ __forceinline__ void plan_tiles(const PlanParams &p, bool keys, bool report, Emit emit, Chunk chunk) {
    const int lane = threadIdx.x & 31;
    for (int s0 = (threadIdx.x >> 5) * 32; s0 < p.num_seqs; s0 += blockDim.x) {
        int q_start = 0, sq = 0, k_start = 0, sk = 0;
        const int seq = s0 + lane;
        bool ok = false;
        if (seq < p.num_seqs) {
            q_start = p.cu_q[seq], sq = p.cu_q[seq + 1] - q_start;
            k_start = p.cu_k[seq], sk = p.cu_k[seq + 1] - k_start;
            const bool q_ok = q_start >= 0 && sq >= 0 && static_cast<int64_t>(q_start) + sq <= p.total_q && sq <= p.max_q;
            const bool k_ok = k_start >= 0 && sk >= 0 && static_cast<int64_t>(k_start) + sk <= p.total_k && sk <= p.max_k;
            if (report && !q_ok) flag_error(p.err, kErrQueryLen);
            if (report && !k_ok) flag_error(p.err, kErrSeqRange);
            ok = q_ok && k_ok;
        }
        const int tiles = ok ? ((keys ? sk : sq) + BM - 1) / BM : 0;
        int end = tiles;  // inclusive sum over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += x;
        }
        const int total = __shfl_sync(0xffffffffu, end, 31);
        if (lane == 0) chunk(s0 / 32, total);
        for (int i0 = 0; i0 < total; i0 += 32) {
            const int i = i0 + lane;
            int src = 0;  // the first lane whose tiles end behind i
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (__shfl_sync(0xffffffffu, end, src + o - 1) <= i) src += o;
            src = min(src, 31);
            const int first = __shfl_sync(0xffffffffu, end - tiles, src);
            const int a = __shfl_sync(0xffffffffu, q_start, src), b = __shfl_sync(0xffffffffu, sq, src);
            const int c = __shfl_sync(0xffffffffu, k_start, src), d = __shfl_sync(0xffffffffu, sk, src);
            if (i < total) emit(s0 / 32, i, i - first, a, b, c, d);
        }
    }
}

__device__ __forceinline__ QTile q_tile(const PlanParams &p, int id, int t, int q_start, int sq, int k_start, int sk) {
    QTile r;
    r.row = q_start + t * BM;
    r.left = sq - t * BM;
    r.pos = sk - sq + t * BM;
    r.k_start = k_start;
    r.sk = sk;
    const int hi = r.pos + min(r.left, BM) - 1;
    r.n = hi < 0 ? 0 : hi / BN - first_key(r.pos, p.window) / BN + 1;
    r.id = id;
    r.pad = 0;
    return r;
}
__device__ __forceinline__ KTile k_tile(const PlanParams &p, int t, int q_start, int sq, int k_start, int sk) {
    KTile r;
    r.row = k_start + t * BM;
    r.left = sk - t * BM;
    r.key = t * BM;
    r.off = sk - sq;
    r.q_start = q_start;
    r.sq = sq;
    const int from = first_query(r);
    int64_t to = sq;
    if (p.window > 0) to = min(to, static_cast<int64_t>(r.key) + min(r.left, BM) - 1 + p.window - r.off);
    r.n = to > from ? static_cast<int>((to - from + BN - 1) / BN) : 0;
    r.from = 0;
    r.to = r.n * p.group;
    r.part = 0;
    r.parts = 1;
    r.slot = 0;
    return r;
}

// Exclusive sums of n numbers in shared memory, by one warp; returns their sum.
__device__ __forceinline__ int exclusive_sums(int *x, int n) {
    const int lane = threadIdx.x & 31;
    int sum = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane, v = i < n ? x[i] : 0;
        int end = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        if (i < n) x[i] = sum + end - v;
        sum += __shfl_sync(0xffffffffu, end, 31);
    }
    return sum;
}

__device__ __forceinline__ void plan_lists(const PlanParams &p) {
    __shared__ __align__(16) int bins[kPlanBins];
    __shared__ int warps[8];  // entries in a warp's bins
    __shared__ int before[65536 / 32];  // tiles of the chunks of 32 sequences before
    __shared__ bool fits;
    __shared__ int slots;
    __shared__ unsigned long long steps;  // of the key tiles, all kv heads
    const int chunks = (p.num_seqs + 31) / 32;
    if (threadIdx.x == 0) slots = 0, steps = 0;
    for (int i = threadIdx.x; i < 8 * p.slots; i += blockDim.x) p.arrived[i] = 0;
    __syncthreads();
    unsigned long long mine = 0;
    plan_tiles(
        p, true, false, [&](int, int, int t, int a, int b, int c, int d) { mine += k_tile(p, t, a, b, c, d).to; }, [](int, int) {});
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if ((threadIdx.x & 31) == 0 && mine > 0) atomicAdd(&steps, mine * p.num_kv_heads);
    __syncthreads();
    const int limit = static_cast<int>(min(steps / kPlanSms + kMinSteps, 1ull << 30));
    // Bins of the list by the number of steps (key tiles: in units of a group's where those would not fit).
    const int unit = p.group * ((p.max_q + BM - 1) / BM) < kPlanBins ? 1 : p.group;
    auto bin = [](int n) { return kPlanBins - 1 - min(n, kPlanBins - 1); };
    // A key tile's parts in turn: fill(entry).
    auto parts_of = [&](KTile x, bool place, auto fill) {
        const int all = x.to;
        x.parts = max((all + limit - 1) / limit, 1);
        const int per = (all + x.parts - 1) / x.parts;  // (at most limit, so no part is empty)
        if (place && x.parts > 1) x.slot = atomicAdd(&slots, x.parts * p.num_kv_heads);
        for (; x.part < x.parts; ++x.part) {
            x.from = x.part * per;
            x.to = min(x.from + per, all);
            fill(x);
        }
    };
    for (int keys = 0; keys < 2; ++keys) {
        for (int i = threadIdx.x; i < kPlanBins; i += blockDim.x) bins[i] = 0;
        __syncthreads();
        plan_tiles(
            p, keys, keys == 0,
            [&](int, int, int t, int a, int b, int c, int d) {
                if (keys)
                    parts_of(k_tile(p, t, a, b, c, d), false, [&](const KTile &x) { atomicAdd(&bins[bin((x.to - x.from + unit - 1) / unit)], 1); });
                else
                    atomicAdd(&bins[bin(q_tile(p, 0, t, a, b, c, d).n)], 1);
            },
            [&](int chunk, int tiles) { before[chunk] = tiles; });
        __syncthreads();
        // (A thread four bins: by one warp the sums of all took 2.5 us.)
        static_assert(kPlanBins == 4 * 256, "four bins a thread");
        int4 &mine4 = reinterpret_cast<int4 *>(bins)[threadIdx.x];
        const int4 n4 = mine4;
        int end = n4.x + n4.y + n4.z + n4.w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, end, o);
            if ((threadIdx.x & 31) >= o) end += x;
        }
        if ((threadIdx.x & 31) == 31) warps[threadIdx.x >> 5] = end;
        __syncthreads();
        int count = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w == threadIdx.x >> 5) end += count;
            count += warps[w];
        }
        mine4 = make_int4(end - n4.x - n4.y - n4.z - n4.w, end - n4.y - n4.z - n4.w, end - n4.z - n4.w, end - n4.w);
        if (threadIdx.x < 32) {
            const int tiles = exclusive_sums(before, chunks);
            if (threadIdx.x == 0) {
                fits = tiles <= p.most[keys];
                p.counts[keys] = fits ? count : 0;
            }
        }
        __syncthreads();
        if (!fits) continue;
        plan_tiles(
            p, keys, false,
            [&](int chunk, int i, int t, int a, int b, int c, int d) {
                if (keys) {
                    parts_of(k_tile(p, t, a, b, c, d), true,
                             [&](const KTile &x) { p.k_list[atomicAdd(&bins[bin((x.to - x.from + unit - 1) / unit)], 1)] = x; });
                } else {
                    const QTile x = q_tile(p, before[chunk] + i, t, a, b, c, d);
                    p.q_list[atomicAdd(&bins[bin(x.n)], 1)] = x;
                }
            },
            [](int, int) {});
        __syncthreads();
    }
}

// Bound by its bytes: 44 us for out and dout of 17400 tokens, 32 heads of 128 (285 MB, 6.5 TB/s).
// lse in base 2 and dout_i out_i, both as [num_heads, total_q]: a block takes 8 tokens of 8 heads, half
// a warp (128 dims) or a quarter (64) a row.  The blocks behind the first write the bias by distance (with a
// launch of its own the smallest training step took 72 us, the host's, instead of 64-69; 64-74 across boxes).  The first block makes
// the lists, for which it spills registers: with the 48 that it would take the others are too few on an SM
// (44 us against 39 for 15000 tokens, 32 heads of 128).
template <int HD>
__global__ void __launch_bounds__(256, 8)
    grad_stat_kernel(const uint4 *__restrict__ out, const uint4 *__restrict__ dout, const float *__restrict__ lse,
                     float *__restrict__ lse2, float *__restrict__ delta, int total_q, int num_heads,
                     const __grid_constant__ PlanParams plan, float *__restrict__ table, const __grid_constant__ RelativeBias bias,
                     int table_blocks) {
    constexpr int LANES = HD / 8, ROWS = 256 / LANES;
    __shared__ float s_l[8][9], s_d[8][9];  // [head][token]
    if (blockIdx.x == 0) {
        if (blockIdx.y == 0) plan_lists(plan);
        return;
    }
    const int h0 = blockIdx.y * 8;
    if (static_cast<int>(blockIdx.x) <= table_blocks) {
        bias_table_entry(table, bias, num_heads, (blockIdx.x - 1) * 256 + threadIdx.x, h0, 1, min(h0 + 8, num_heads));
        return;
    }
    const int t0 = (blockIdx.x - 1 - table_blocks) * 8;
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
            s_l[r % 8][r / 8] = e < kNoDigits ? INFINITY : e * kLog2e;
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
    using L = LayoutQ<HD, BIAS>;
    constexpr int NR = L::NR, NA = L::NA, NB = L::NB;
    constexpr uint32_t kDp = 128, kDq = 384;
    if constexpr (BIAS) {  // the buckets' first distances, behind the rows' sums
        extern __shared__ __align__(1024) uint8_t smem_raw[];
        int *first = reinterpret_cast<int *>(smem_raw + L::OFF_SMALL) + kFirstAt;
        for (int i = threadIdx.x; i <= p.bias.num_buckets; i += kThreads) first[i] = p.bias.first[i];
    }
    const Cta c = setup<L>(1);
    auto bar = [&](int i) -> uint32_t { return c.base + L::OFF_BAR + 8u * static_cast<uint32_t>(i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto sQ = [&](uint32_t slot) -> uint32_t { return c.base + L::OFF_RES + slot * 2 * L::TILE; };
    auto sDo = [&](uint32_t slot) -> uint32_t { return sQ(slot) + L::TILE; };
    auto sK = [&](uint32_t st) -> uint32_t { return c.base + L::OFF_A + st * L::TILE; };
    auto sV = [&](uint32_t st) -> uint32_t { return c.base + L::OFF_B + st * L::TILE; };
    const int last = p.bias.last();
    const uint32_t table_bytes = BIAS ? near_entries(last) * 4u : 0u;
    const bool table_here = BIAS && table_bytes <= kTableBytesQ;
    const int count = *p.counts;
    // An item's steps: the tiles 0 .. n_pre - 1 with D from dout . out; tiles n_pre .. n - 2 for D alone;
    // the last tile, where D is complete before its dS is formed; then tiles n_pre .. n - 2 with D.
    // In the second pass, over the items that are done again, all tiles with D.
    struct Steps {
        int n, n_far, n_pre, n_all, kt0;
        __device__ int tile(int j) const { return j < n ? j : j - (n - n_pre); }
        __device__ bool sum_only(int j) const { return j >= n_pre && j + 1 < n; }
        __device__ bool first_dq(int j) const { return j == (n_pre > 0 ? 0 : n - 1); }
    };
    auto steps_of = [&](const QTile &t, int pass) -> Steps {
        Steps s;
        const int kmin = first_key(t.pos, p.window);
        s.n = t.n;
        s.kt0 = kmin / BN;
        // (tiles of the last bucket alone)
        s.n_far = BIAS ? min(max(kmin, t.pos - last + 1) / BN - s.kt0, t.n) : t.n;
        const bool few = t.pos + 1 < kFewKeys || (p.window > 0 && p.window < kFewKeys);
        s.n_pre = pass > 0 ? t.n : few ? 0 : s.n_far;
        s.n_all = s.n + max(s.n - 1 - s.n_pre, 0);
        return s;
    };
    // Between the passes the roles meet: all of the block's items have their D, and whether they are done again is known.
    auto second_pass = [&]() -> bool {
        asm volatile("bar.sync 1, 352;" ::: "memory");
        return *c.again != 0 && *c.abort_flag == 0;
    };
    auto first_item = [&](int pass) -> int { return pass > 0 ? next_again(0, count, p.num_heads, p.again) : 0; };
    auto item_after = [&](int k, int pass) -> int { return pass > 0 ? next_again(k + 1, count, p.num_heads, p.again) : k + 1; };

    // With a bias, registers go from the warps that load and issue to the element-wise ones, which spill with
    // 168 (304 us against 293 for 16 sequences of 128-2048 tokens, 32/8 heads; without a bias the split costs
    // two documents of 6000-8192 tokens 12 us of 664): 384 threads of 168 are 256 of 208 and 128 of 88.
    if (warp >= 8) {
        if constexpr (BIAS) setmaxnreg_dec<88>();
        if (warp == kWarpLoad) {
            if (lane < 4) prefetch_tmap(lane == 0 ? p.tmap_q : lane == 1 ? p.tmap_do : lane == 2 ? p.tmap_k : p.tmap_v);
            uint32_t lands = 0, items = 0, J = 0, sa = 0, pa = 1;  // ring A: stage, phase of its emptying
            bool ok = true;
            int e, h;
            for (int pass = 0; pass < 2; ++pass) {
                if (pass > 0 && !second_pass()) break;
                for (int k = first_item(pass); ok && item_of(k, count, p.num_heads, e, h); k = item_after(k, pass)) {
                    const QTile t = load_entry(p.q_list, e);
                    if (t.n == 0) continue;
                    const Steps s = steps_of(t, pass);
                    const uint32_t res = items % NR;
                    if (items >= NR && !wait_warp(bar(res_empty(res)), (items / NR - 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
                    // (Sums along diagonals run across rows; in all else a row behind the sequence stays on its own.)
                    const bool edit = BIAS && ragged(t.left);
                    const uint32_t land = bar(edit ? B_LAND : res_full(res));
                    if (lane == 0) mbar_arrive_expect_tx(land, 2 * L::TILE);
                    __syncwarp();
                    load_tile<HD>(p.tmap_q, sQ(res), h, t.row, 0, t.left, land);
                    load_tile<HD>(p.tmap_do, sDo(res), h, t.row, 0, t.left, land);
                    if (edit) {
                        if (!wait_warp(land, lands++ & 1, c.abort_flag, p.err, kTimeoutNs)) break;
                        clear_rows<HD>(sQ(res), t.left);
                        clear_rows<HD>(sDo(res), t.left);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(res_full(res)));
                    }
                    if (table_here) {
                        const uint32_t slot = items & 1;
                        if (items >= 2 && !wait_warp(bar(B_TABFREE + slot), ((items >> 1) - 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar(B_TABFULL + slot), table_bytes);
                            bulk_load(c.base + L::OFF_SMALL + kSmallQBias + slot * kTableBytesQ, bias_row_of(p.bias_table, h, last) - kNearPad,
                                      table_bytes, bar(B_TABFULL + slot));
                        }
                        __syncwarp();
                    }
                    ++items;
                    const int kvh = h / p.group;
                    for (int j = 0; j < s.n_all; ++j, ++J) {
                        const uint32_t sb = J % NB, full_k = bar(B_AFULL + sa), full_v = bar(B_BFULL + sb);
                        const int row0 = (s.kt0 + s.tile(j)) * BN;
                        const bool cut = ragged(t.sk - row0);  // (the copies of tiles that are edited land together)
                        ok = J < NA || wait_warp(bar(B_AEMPTY + sa), pa, c.abort_flag, p.err, kTimeoutNs);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(cut ? bar(B_LAND) : full_k, cut ? 2 * L::TILE : L::TILE);
                        __syncwarp();
                        load_tile<HD>(p.tmap_k, sK(sa), kvh, t.k_start, row0, t.sk, cut ? bar(B_LAND) : full_k);
                        ok = J < NB || wait_warp(bar(B_BEMPTY + sb), (J / NB - 1) & 1, c.abort_flag, p.err, kTimeoutNs);
                        if (!ok) break;
                        if (lane == 0 && !cut) mbar_arrive_expect_tx(full_v, L::TILE);
                        __syncwarp();
                        load_tile<HD>(p.tmap_v, sV(sb), kvh, t.k_start, row0, t.sk, cut ? bar(B_LAND) : full_v);
                        if (cut) {
                            ok = wait_warp(bar(B_LAND), lands++ & 1, c.abort_flag, p.err, kTimeoutNs);
                            if (!ok) break;
                            clear_rows<HD>(sK(sa), t.sk - row0);
                            clear_rows<HD>(sV(sb), t.sk - row0);
                            __syncwarp();
                            if (lane == 0) mbar_arrive(full_k), mbar_arrive(full_v);
                        }
                        if (++sa == NA) sa = 0, pa ^= 1u;
                    }
                }
            }
        } else if (warp == kWarpMma || warp == kWarpMma2) {
            // One warp issues S and dP, the other dQ, so that neither's waits hold up the other's products.
            // The whole warp waits, one lane issues (always the same: a commit covers what its thread issued).
            auto wait = [&](int b, uint32_t parity) {
                const bool ok = wait_warp(bar(b), parity, c.abort_flag, p.err, kTimeoutNs);
                tc_fence_after();
                return ok;
            };
            uint32_t items = 0, J = 0, sa = 0, pa = 0;  // stage of ring A and its phase
            bool ok = true;
            int e, h;
            for (int pass = 0; pass < 2; ++pass) {
                if (pass > 0 && !second_pass()) break;
                for (int k = first_item(pass); ok && item_of(k, count, p.num_heads, e, h); k = item_after(k, pass)) {
                    const QTile t = load_entry(p.q_list, e);
                    if (t.n == 0) continue;
                    const Steps s = steps_of(t, pass);
                    if (warp == kWarpMma) {
                        const uint32_t res = items % NR;
                        ok = wait(res_full(res), (items / NR) & 1);
                        for (int j = 0; ok && j < s.n_all; ++j, ++J) {
                            const uint32_t sb = J % NB, sd = J & 1;  // stage of V, place of dP
                            ok = wait(B_AFULL + sa, pa) && (J == 0 || wait(B_PFULL, (J - 1) & 1));
                            if (!ok) break;
                            if (elect_one()) {
                                issue_abt<HD>(c.tmem, sQ(res), sK(sa));
                                mma_commit(bar(B_SFULL));
                            }
                            __syncwarp();
                            // (dP goes where dS of the step before the last one was: its dQ has to be done.)
                            ok = wait(B_BFULL + sb, (J / NB) & 1) && (J < 2 || wait(B_DQDONE + sd, ((J >> 1) - 1) & 1));
                            if (!ok) break;
                            if (elect_one()) {
                                issue_abt<HD>(c.tmem + kDp + 128u * sd, sDo(res), sV(sb));
                                mma_commit(bar(B_DPFULL + sd));
                                mma_commit(bar(B_BEMPTY + sb));
                                if (j + 1 == s.n_all) mma_commit(bar(res_empty(res)));
                            }
                            __syncwarp();
                            if (++sa == NA) sa = 0, pa ^= 1u;
                        }
                    } else {
                        for (int j = 0; j < s.n_all; ++j, ++J) {
                            const bool first = s.first_dq(j);
                            ok = wait(B_DSFULL + (J & 1), (J >> 1) & 1) && (!first || items == 0 || wait(B_ACCFREE, (items - 1) & 1));
                            if (!ok) break;
                            if (elect_one()) {
                                if (!s.sum_only(j)) issue_ab<HD>(c.tmem + kDq, c.tmem + kDp + 128u * (J & 1), sK(sa), first);
                                mma_commit(bar(B_DQDONE + (J & 1)));
                                mma_commit(bar(B_AEMPTY + sa));
                                if (j + 1 == s.n_all) mma_commit(bar(B_DONE));
                            }
                            __syncwarp();
                            if (++sa == NA) sa = 0;
                        }
                    }
                    ++items;
                }
            }
        }
    } else {
        if constexpr (BIAS) setmaxnreg_inc<208>();
        const int wg = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;  // (of D and dQ)
        const int r0 = quarter * 32 + (lane >> 2), c0 = lane & 3;  // first row of the block, columns 2 c0, 2 c0 + 1
        const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
        const float sl2 = p.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        float *small = reinterpret_cast<float *>(c.sb + L::OFF_SMALL);
        [[maybe_unused]] const int *first = reinterpret_cast<const int *>(small) + kFirstAt;
        const bool v8 = aligned32(p.dq, p.dq_stride);
        uint32_t items = 0, J = 0;
        bool ok = true;
        int next_entry, next_head;
        QTile next{};
        float next_lse[4] = {}, next_delta[4] = {}, next_far = 0.f;
        auto prefetch = [&] {  // what the next item needs of its rows and its head
            next = load_entry(p.q_list, next_entry);
            const int64_t at = static_cast<int64_t>(next_head) * p.total_q + next.row;
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int x = r0 + 8 * a;
                next_lse[a] = x < next.left ? p.lse2[at + x] : INFINITY;
                next_delta[a] = x < next.left ? p.delta[at + x] : 0.f;
            }
            if (BIAS) next_far = __ldg(bias_row_of(p.bias_table, next_head, last) - kBiasPad);
        };
        for (int pass = 0; pass < 2; ++pass) {
            if (pass > 0 && !second_pass()) break;
            int k = first_item(pass);
            bool more = ok && item_of(k, count, p.num_heads, next_entry, next_head);
            if (more) prefetch();
            while (ok && more) {
                const QTile t = next;
                const int head = next_head;
                // (wg 0) where it says whether the item is done again
                uint8_t *const again = p.again + (static_cast<int64_t>(next_entry) * p.num_heads + head) * 4 + quarter;
                float lse2[4], delta[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) lse2[a] = next_lse[a], delta[a] = next_delta[a];
                [[maybe_unused]] const float last_bias = next_far;
                k = item_after(k, pass);
                more = item_of(k, count, p.num_heads, next_entry, next_head);
                const int rows = min(t.left, BM);
                const int64_t stat_row = static_cast<int64_t>(head) * p.total_q + t.row;
                __nv_bfloat16 *dq = p.dq + static_cast<int64_t>(t.row) * p.dq_stride + head * HD;
                [[maybe_unused]] float by_bucket[4] = {0.f, 0.f, 0.f, 0.f};
                float *partial = nullptr;
                if constexpr (BIAS)
                    partial = p.partial + ((static_cast<int64_t>(t.id) * p.num_heads + head) * 8 + warp) * p.bias.num_buckets;
                if (t.n == 0) {
                    zero_rows<HD>(dq, p.dq_stride, rows);
                    if (wg == 0 && row < rows) p.delta[stat_row + row] = 0.f;
                    if (wg == 0 && lane == 0) *again = 0;
                    if constexpr (BIAS)
                        for (int b = lane; b < p.bias.num_buckets; b += 32) partial[b] = 0.f;
                    if (more) prefetch();
                    continue;
                }
                const Steps s = steps_of(t, pass);
                float d_sum[4] = {0.f, 0.f, 0.f, 0.f}, abs_sum[4] = {0.f, 0.f, 0.f, 0.f};  // of P dP, of |dS| with dout . out
                // Sums of P dP and of P over the first n_far tiles (d_far: and of the last bucket's dS in the others).
                [[maybe_unused]] float d_far = 0.f, w_far[4] = {0.f, 0.f, 0.f, 0.f};
                [[maybe_unused]] const float *bias_row = nullptr;  // entry of distance 0
                if constexpr (BIAS) {
                    bias_row = bias_row_of(p.bias_table, head, last);
                    if (table_here) {
                        ok = wait_warp(bar(B_TABFULL + (items & 1)), (items >> 1) & 1, c.abort_flag, p.err, kTimeoutNs);
                        if (!ok) break;
                        bias_row = small + kSmallQBias / 4 + (items & 1) * (kTableBytesQ / 4) + kNearPad;
                    }
                }
                bool moved = false;  // (wg 0) dout . out moved a row of the warp too far
                for (int j = 0; j < s.n_all; ++j, ++J) {
                    const uint32_t dp = c.tmem + t_lane + kDp + 128u * (J & 1) + 64u * wg;
                    const bool sum_only = s.sum_only(j);
                    const int tile = s.tile(j);
                    ok = wait_warp(bar(B_SFULL), J & 1, c.abort_flag, p.err, kTimeoutNs);
                    if (!ok) break;
                    tc_fence_after();
                    float w[2][32];  // logits, then weights P
                    load_block(c.tmem + t_lane + 64u * wg, w);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_PFULL));
                    // The distance of the warp's first row to its first key: its block has d00 - 63 .. d00 + 31.
                    const int d00 = t.pos + quarter * 32 - (s.kt0 + tile) * BN - 64 * wg;
                    const bool near = BIAS && d00 - 63 < last;
                    const float add = BIAS ? near ? bias_ref(last_bias) : last_bias : 0.f;
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const float x = add - lse2[a];
                        const uint64_t x2 = f2_pack(x, x);
#pragma unroll
                        for (int b = 0; b < 8; ++b) set_pair(w, a, b, f2_fma(block_pair(w, a, b), sl2x2, x2));
                    }
                    if (near || (!BIAS && d00 < 63) || (p.window > 0 && d00 + 31 >= p.window)) {
                        const int n0 = d00 + (lane >> 2) - 2 * c0 - 56;
                        auto entry = [&](int n) -> float {
                            float x = 0.f;
                            if (near)
                                x = bias_row[n];  // (-inf before distance 0)
                            else if (!BIAS && n < 0)
                                x = -INFINITY;
                            return p.window > 0 && n >= p.window ? -INFINITY : x;
                        };
#pragma unroll
                        for (int g = 0; g < 11; ++g) {  // a - b + 7
                            const uint64_t x2 = f2_pack(entry(n0 + 8 * g), entry(n0 + 8 * g - 1));
#pragma unroll
                            for (int a = 0; a < 4; ++a) {
                                const int b = a + 7 - g;
                                if (b >= 0 && b < 8) set_pair(w, a, b, f2_add(block_pair(w, a, b), x2));
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 64; ++i) w[i >> 5][i & 31] = ex2_approx(w[i >> 5][i & 31]);
                    if (BIAS && !sum_only && tile < s.n_far) {
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            uint64_t x = block_pair(w, a, 0);
#pragma unroll
                            for (int b = 1; b < 8; ++b) x = f2_add(x, block_pair(w, a, b));
                            w_far[a] += pair_sum(x);
                        }
                    }
                    ok = wait_warp(bar(B_DPFULL + (J & 1)), (J >> 1) & 1, c.abort_flag, p.err, kTimeoutNs);
                    if (!ok) break;
                    tc_fence_after();
                    // D of the rows: a thread's columns, its four threads', this warpgroup's half and the other's.
                    auto exchange = [&]() -> bool {
                        const bool odd = c0 & 1, high = c0 & 2;
                        auto own = [&](const float (&f)[4]) -> float {  // that of the thread's row r0 + 8 c0
                            return high ? (odd ? f[3] : f[2]) : (odd ? f[1] : f[0]);
                        };
                        auto across = [&](const float (&f)[4]) -> float {
                            const float x0 = (odd ? f[1] : f[0]) + __shfl_xor_sync(0xffffffffu, odd ? f[0] : f[1], 1);
                            const float x1 = (odd ? f[3] : f[2]) + __shfl_xor_sync(0xffffffffu, odd ? f[2] : f[3], 1);
                            return (high ? x1 : x0) + __shfl_xor_sync(0xffffffffu, high ? x0 : x1, 2);
                        };
                        // (Two places: a warpgroup may be an item ahead of the other's reading.)
                        float *sums = small + 256 * (items & 1);
                        __nv_bfloat16 *abs_of = reinterpret_cast<__nv_bfloat16 *>(small + kAbsAt) + 128 * (items & 1);
                        [[maybe_unused]] __nv_bfloat16 *weight_of = reinterpret_cast<__nv_bfloat16 *>(small + kWeightAt) + 128 * (items & 1);
                        const int x = r0 + 8 * c0;
                        sums[128 * wg + x] = across(d_sum);
                        float abs_all = across(abs_sum);
                        [[maybe_unused]] float weight = 1.f;
                        if constexpr (BIAS) weight = across(w_far);
                        if (wg == 1) {
                            abs_of[x] = __float2bfloat16_rd(abs_all);
                            if constexpr (BIAS) weight_of[x] = __float2bfloat16_ru(weight);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_SUMS));
                        if (!wait_warp(bar(B_SUMS), items & 1, c.abort_flag, p.err, kTimeoutNs)) return false;
                        const float before = own(delta);
#pragma unroll
                        for (int a = 0; a < 4; ++a) delta[a] = sums[r0 + 8 * a] + sums[128 + r0 + 8 * a];
                        if (wg == 0) {
                            const float d = own(delta);
                            if (x < rows) p.delta[stat_row + x] = d;
                            abs_all += __bfloat162float(abs_of[x]);
                            if constexpr (BIAS) weight += __bfloat162float(weight_of[x]);
                            const bool off = s.n_pre > 0 && x < rows && fabsf(d - before) * weight > kMoved * abs_all;
                            moved = __any_sync(0xffffffffu, off);
                        }
                        return true;
                    };
                    const bool pivot = j + 1 == s.n && s.n_pre < s.n;
                    if (pivot) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float d[32];
                            tmem_ld_16x256b_x8(dp + static_cast<uint32_t>(half * 16 << 16), d);
                            tmem_wait_ld_regs(d);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int a = 2 * half + u;
                                uint64_t x = 0ull;
#pragma unroll
                                for (int b = 0; b < 8; ++b)
                                    x = f2_fma(block_pair(w, a, b), f2_pack(d[pair_at(a, b)], d[pair_at(a, b) + 1]), x);
                                d_sum[a] += pair_sum(x);
                            }
                        }
                        ok = exchange();
                        if (!ok) break;
                        if (s.n_pre == 0) {  // (the last bucket's tiles may still be to come)
#pragma unroll
                            for (int a = 0; a < 4; ++a) d_sum[a] = 0.f;
                        }
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float d[32];
                        tmem_ld_16x256b_x8(dp + static_cast<uint32_t>(half * 16 << 16), d);
                        tmem_wait_ld_regs(d);
                        uint32_t pk[16];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int a = 2 * half + u;
                            const uint64_t delta2 = f2_pack(-delta[a], -delta[a]);
                            uint64_t x = 0ull;
#pragma unroll
                            for (int b = 0; b < 8; ++b) {
                                const uint64_t w2 = block_pair(w, a, b), d2 = f2_pack(d[pair_at(a, b)], d[pair_at(a, b) + 1]);
                                x = f2_fma(w2, d2, x);
                                set_pair(w, a, b, f2_mul(w2, f2_add(d2, delta2)));
                                pk[2 * b + u] = pack_bf16x2(w[half][pair_at(a, b)], w[half][pair_at(a, b) + 1]);
                            }
                            if (!pivot) d_sum[a] += pair_sum(x);
                        }
                        if (!sum_only) tmem_st_16x128b_x8(dp + static_cast<uint32_t>(half * 16 << 16), pk);
                    }
                    if (!sum_only) {
                        if (BIAS && tile + 1 == s.n_far) d_far += (d_sum[0] + d_sum[1]) + (d_sum[2] + d_sum[3]);
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_DSFULL + (J & 1)));
                    if (pass == 0 && j < s.n_pre) {
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            float x = 0.f, y = 0.f;
#pragma unroll
                            for (int b = 0; b < 8; ++b) {
                                x += fabsf(w[a >> 1][pair_at(a, b)]);
                                y += fabsf(w[a >> 1][pair_at(a, b) + 1]);
                            }
                            abs_sum[a] += x + y;
                        }
                    }
                    if (pass == 0 && j + 1 == s.n && s.n_pre == s.n) {
                        ok = exchange();
                        if (!ok) break;
                    }
                    if (BIAS && pass == 0 && j + 1 >= s.n && tile >= s.n_far && d00 > -32) {  // (else all of the block is hidden)
                        // Sums along diagonals: a thread's own, 11 pairs; then thread (r, c), r = t / 4, fetches of the
                        // threads (., c) those of distances r + 8 i (v[i], less d00 - 64); then the four threads of
                        // an r share them out.
                        float v[12];
#pragma unroll
                        for (int i = 0; i < 12; ++i) v[i] = 0.f;
#pragma unroll
                        for (int g = 0; g < 11; ++g) {
                            uint64_t x2 = 0ull;
#pragma unroll
                            for (int a = 0; a < 4; ++a) {
                                const int b = a + 7 - g;
                                if (b >= 0 && b < 8) x2 = f2_add(x2, block_pair(w, a, b));
                            }
                            float x[2];
                            f2_unpack(x2, x[0], x[1]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int src = (lane >> 2) + 2 * c0 + k;
                                const float y = __shfl_sync(0xffffffffu, x[k], (src & 7) * 4 + c0);
                                if (src >= 8)
                                    v[g] += y;
                                else
                                    v[g + 1] += y;
                            }
                        }
                        const int base = d00 - 64;
                        float *diag = small + kDiagAt + 96 * warp;
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            float x[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float even = v[4 * k + 2 * i], odd = v[4 * k + 2 * i + 1];
                                x[i] = (c0 & 1 ? odd : even) + __shfl_xor_sync(0xffffffffu, c0 & 1 ? even : odd, 1);
                            }
                            const float y = (c0 & 2 ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, c0 & 2 ? x[0] : x[1], 2);
                            const int at = (lane >> 2) + 8 * c0 + 32 * k;
                            diag[at] = y;
                            if (base + at >= last) d_far += y;
                        }
                        __syncwarp();
                        // A lane adds up the distances of its buckets.  (Scans over the warp's 96 distances by bucket
                        // took 60 us of 375 of sixteen sequences of 128-2048 tokens.)
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            if (32 * k4 >= p.bias.num_buckets - 1) break;
                            const int b = lane + 32 * k4;
                            if (b >= p.bias.num_buckets - 1) continue;
                            const int hi = min(first[b + 1] - base, 96);
                            float sum = 0.f;
#pragma unroll 1
                            for (int x = max(first[b] - base, 0); x < hi; x += 4) {
                                float f[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) f[i] = x + i < hi ? diag[x + i] : 0.f;
                                sum += (f[0] + f[1]) + (f[2] + f[3]);
                            }
                            by_bucket[k4] += sum;
                        }
                        __syncwarp();
                    }
                }
                if (!ok) break;
                if constexpr (BIAS) {
                    __syncwarp();
                    if (table_here && lane == 0) mbar_arrive(bar(B_TABFREE + (items & 1)));
                    if (pass == 0) {
                        const float t_far = warp_sum(d_far - ((delta[0] * w_far[0] + delta[1] * w_far[1]) + (delta[2] * w_far[2] + delta[3] * w_far[3])));
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            const int b = lane + 32 * k4;
                            if (b < p.bias.num_buckets) partial[b] = by_bucket[k4] + (b == p.bias.num_buckets - 1 ? t_far : 0.f);
                        }
                    }
                }
                if (pass == 0 && wg == 0 && lane == 0) {
                    *again = moved;
                    if (moved) *c.again = 1;
                }
                if (more) prefetch();
                ok = wait_warp(bar(B_DONE), items & 1, c.abort_flag, p.err, kTimeoutNs);
                if (!ok) break;
                tc_fence_after();
                __nv_bfloat16 *dst = dq + static_cast<int64_t>(row) * p.dq_stride + wg * (HD / 2);
#pragma unroll 1
                for (int cc = 0; cc < HD / 64; ++cc)
                    store_chunk(c.tmem + t_lane + kDq + wg * (HD / 2) + cc * 32, p.scale, dst + cc * 32, row < rows, v8);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_ACCFREE));
                ++items;
            }
        }
    }
    teardown(c);
}

// --------------------------------------------------------------------- dK, dV ---
// Tensor memory: S^T (then P^T) at 0, dP^T (then dS^T) at 128, dV at 256, dK at 384.  While the
// element-wise warps form P^T, the tensor cores run dK of the tile before and dP^T; while they form
// dS^T, dV and the next tile's S^T:
//     dP(i), dV(i), S(i + 1), dK(i).
template <int HD, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) grad_kv_kernel(const __grid_constant__ GradParams p) {
    using L = LayoutKv<HD, BIAS>;
    constexpr int NR = L::NR;
    constexpr uint32_t kS = 0, kDp = 128, kDv = 256, kDk = 384;
    const Cta c = setup<L>(2);
    auto bar = [&](int i) -> uint32_t { return c.base + L::OFF_BAR + 8u * static_cast<uint32_t>(i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto sK = [&](uint32_t slot) -> uint32_t { return c.base + L::OFF_RES + slot * 2 * L::TILE; };
    auto sV = [&](uint32_t slot) -> uint32_t { return sK(slot) + L::TILE; };
    auto sQ = [&](int st) -> uint32_t { return c.base + L::OFF_A + st * L::TILE; };
    auto sDo = [&](int st) -> uint32_t { return c.base + L::OFF_B + st * L::TILE; };
    // Per stage and query of the tile: -lse2 (BIAS: plus what the table is relative to), -D and (BIAS) the
    // last bucket's bias - lse2.
    auto stat = [&](int st) -> float * { return reinterpret_cast<float *>(c.sb + L::OFF_SMALL) + st * 384; };
    const int last = p.bias.last();

    const uint32_t head_bytes = BIAS ? near_entries(last) * 4u : 0u, table_bytes = head_bytes * p.group;
    const bool table_here = BIAS && table_bytes <= kTableBytes;
    const int count = p.counts[1];

    if (warp == kWarpLoad) {
        if (lane < 4) prefetch_tmap(lane == 0 ? p.tmap_q : lane == 1 ? p.tmap_do : lane == 2 ? p.tmap_k : p.tmap_v);
        uint32_t lands = 0, items = 0, J = 0;
        bool ok = true;
        int e, kvh;
        for (int k = 0; ok && item_of(k, count, p.num_kv_heads, e, kvh); ++k) {
            const KTile t = load_entry(p.k_list, e);
            if (t.n == 0) continue;
            const uint32_t res = items % NR;
            if (items >= NR && !wait_warp(bar(res_empty(res)), (items / NR - 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(res_full(res)), 2 * L::TILE);
            __syncwarp();
            load_tile<HD>(p.tmap_k, sK(res), kvh, t.row, 0, t.left, bar(res_full(res)));
            load_tile<HD>(p.tmap_v, sV(res), kvh, t.row, 0, t.left, bar(res_full(res)));
            if (table_here) {
                const uint32_t slot = items & 1;
                if (items >= 2 && !wait_warp(bar(B_TABFREE + slot), ((items >> 1) - 1) & 1, c.abort_flag, p.err, kTimeoutNs)) break;
                if (lane == 0) mbar_arrive_expect_tx(bar(B_TABFULL + slot), table_bytes);
                __syncwarp();
                for (int g = lane; g < p.group; g += 32)
                    bulk_load(c.base + L::OFF_SMALL + kSmallKv + slot * kTableBytes + g * head_bytes,
                              bias_row_of(p.bias_table, kvh * p.group + g, last) - kNearPad, head_bytes, bar(B_TABFULL + slot));
                __syncwarp();
            }
            ++items;
            const int r_first = first_query(t);
            for (int i = t.from; ok && i < t.to; ++i, ++J) {
                const uint32_t st = J & 1;
                const int r = r_first + i % t.n * BN, head = kvh * p.group + i / t.n;
                // (dout's stage is free first: dV comes before dK.  The copies of a tile that is edited
                // are under way together.)
                const bool cut = ragged(t.sq - r);
                const uint32_t full = bar(B_AFULL + st), land = cut ? bar(B_LAND) : full;
                ok = J < 2 || wait_warp(bar(B_BEMPTY + st), ((J >> 1) - 1) & 1, c.abort_flag, p.err, kTimeoutNs);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(land, 2 * L::TILE);
                __syncwarp();
                load_tile<HD>(p.tmap_do, sDo(st), head, t.q_start, r, t.sq, land);
                ok = J < 2 || wait_warp(bar(B_AEMPTY + st), ((J >> 1) - 1) & 1, c.abort_flag, p.err, kTimeoutNs);
                if (!ok) break;
                load_tile<HD>(p.tmap_q, sQ(st), head, t.q_start, r, t.sq, land);
                float far = 0.f, ref = 0.f;
                if constexpr (BIAS) {
                    far = __ldg(bias_row_of(p.bias_table, head, last) - kBiasPad);
                    ref = bias_ref(far);
                }
                const int64_t at = static_cast<int64_t>(head) * p.total_q + t.q_start + r;
#pragma unroll
                for (int x4 = 0; x4 < 4; ++x4) {
                    const int x = lane + 32 * x4;
                    const bool in = r + x < t.sq;
                    const float l2 = in ? p.lse2[at + x] : INFINITY;
                    stat(st)[x] = ref - l2;
                    stat(st)[128 + x] = in ? -p.delta[at + x] : 0.f;
                    if constexpr (BIAS) stat(st)[256 + x] = far - l2;
                }
                if (cut) {
                    ok = wait_warp(land, lands++ & 1, c.abort_flag, p.err, kTimeoutNs);
                    if (!ok) break;
                    clear_rows<HD>(sDo(st), t.sq - r);
                    clear_rows<HD>(sQ(st), t.sq - r);
                }
                __syncwarp();
                if (lane == 0) {
                    if (cut) mbar_arrive(full);
                    mbar_arrive(full);
                }
            }
        }
    } else if (warp == kWarpMma) {
        auto wait = [&](int b, uint32_t parity) {
            const bool ok = wait_warp(bar(b), parity, c.abort_flag, p.err, kTimeoutNs);
            tc_fence_after();
            return ok;
        };
        uint32_t items = 0, J = 0;
        bool ok = true;
        int e, kvh;
        for (int k = 0; ok && item_of(k, count, p.num_kv_heads, e, kvh); ++k) {
            const KTile t = load_entry(p.k_list, e);
            const int n = t.to - t.from;
            if (n == 0) continue;
            const uint32_t res = items % NR;
            ok = wait(res_full(res), (items / NR) & 1) && wait(B_AFULL + (J & 1), (J >> 1) & 1);
            if (!ok) break;
            if (elect_one()) {
                issue_abt<HD>(c.tmem + kS, sK(res), sQ(J & 1));
                mma_commit(bar(B_SFULL));
            }
            __syncwarp();
            for (int i = 0; i < n; ++i, ++J) {
                const uint32_t st = J & 1, sn = st ^ 1u;
                if (elect_one()) {
                    issue_abt<HD>(c.tmem + kDp, sV(res), sDo(st));
                    mma_commit(bar(B_DPFULL));
                    if (i + 1 == n) mma_commit(bar(res_empty(res)));
                }
                __syncwarp();
                // (The item before's accumulators are stored before they are overwritten.)
                ok = wait(B_PFULL, J & 1) && (i > 0 || items == 0 || wait(B_ACCFREE, (items - 1) & 1));
                if (!ok) break;
                if (elect_one()) {
                    issue_ab<HD>(c.tmem + kDv, c.tmem + kS, sDo(st), i == 0);
                    mma_commit(bar(B_BEMPTY + st));
                }
                __syncwarp();
                if (i + 1 < n) {
                    ok = wait(B_AFULL + sn, ((J + 1) >> 1) & 1);
                    if (!ok) break;
                    if (elect_one()) {
                        issue_abt<HD>(c.tmem + kS, sK(res), sQ(sn));
                        mma_commit(bar(B_SFULL));
                    }
                    __syncwarp();
                }
                ok = wait(B_DSFULL, J & 1);
                if (!ok) break;
                if (elect_one()) {
                    issue_ab<HD>(c.tmem + kDk, c.tmem + kDp, sQ(st), i == 0);
                    mma_commit(bar(B_AEMPTY + st));
                    if (i + 1 == n) mma_commit(bar(B_DONE));
                }
                __syncwarp();
            }
            ++items;
        }
    } else if (warp < 8) {
        const int wg = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
        const float sl2 = p.scale_log2;
        const int c0 = lane & 3;  // columns 2 c0, 2 c0 + 1
        const uint32_t sc = c.tmem + t_lane + kS + 64u * wg, dp = c.tmem + t_lane + kDp + 64u * wg;
        uint32_t items = 0, J = 0;
        bool ok = true;
        int next_entry, next_kvh;
        bool more = item_of(0, count, p.num_kv_heads, next_entry, next_kvh);
        KTile next{};
        if (more) next = load_entry(p.k_list, next_entry);
        for (int k = 0; ok && more; ++k) {
            const KTile t = next;
            const int kvh = next_kvh;  // (the place of a split tile's sums goes by it, at the item's end)
            const int head0 = kvh * p.group;
            const int rows = min(t.left, BM);
            __nv_bfloat16 *dk = p.dk + static_cast<int64_t>(t.row) * p.dk_stride + kvh * HD;
            __nv_bfloat16 *dv = p.dv + static_cast<int64_t>(t.row) * p.dv_stride + kvh * HD;
            more = item_of(k + 1, count, p.num_kv_heads, next_entry, next_kvh);
            if (more) next = load_entry(p.k_list, next_entry);
            if (t.n == 0) {  // no row sees these keys
                zero_rows<HD>(dk, p.dk_stride, rows);
                zero_rows<HD>(dv, p.dv_stride, rows);
                continue;
            }
            const int pos_first = t.off + first_query(t) + 64 * wg;  // of this warpgroup's first query
            [[maybe_unused]] const float *bias_row = nullptr;  // entry of distance 0 of the item's first head
            [[maybe_unused]] int bias_step = bias_stride(last);  // to the next head's
            if constexpr (BIAS) {
                bias_row = bias_row_of(p.bias_table, head0, last);
                if (table_here) {
                    ok = wait_warp(bar(B_TABFULL + (items & 1)), (items >> 1) & 1, c.abort_flag, p.err, kTimeoutNs);
                    if (!ok) break;
                    bias_row = reinterpret_cast<const float *>(c.sb + L::OFF_SMALL + kSmallKv + (items & 1) * kTableBytes) + kNearPad;
                    bias_step = head_bytes / 4;
                }
            }
            for (int i = t.from, g = t.from / t.n, q = t.from % t.n; i < t.to; ++i, ++J) {
                const uint32_t st = J & 1;
                const int pos0 = pos_first + q * BN;
                if (!wait_warp(bar(B_AFULL + st), (J >> 1) & 1, c.abort_flag, p.err, kTimeoutNs) ||
                    !wait_warp(bar(B_SFULL), J & 1, c.abort_flag, p.err, kTimeoutNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float w[2][32];
                load_block(sc, w);
                // The distance of the first query to the warp's first key: its block has d00 - 31 .. d00 + 63.
                const int d00 = pos0 - t.key - quarter * 32;
                const bool near = BIAS && d00 - 31 < last;
                const uint64_t sl2x2 = f2_pack(sl2, sl2);
                const float *nl = stat(st) + (BIAS && !near ? 256 : 0) + 64 * wg + 2 * c0;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const uint64_t l2 = *reinterpret_cast<const uint64_t *>(nl + 8 * b);
#pragma unroll
                    for (int a = 0; a < 4; ++a) set_pair(w, a, b, f2_fma(block_pair(w, a, b), sl2x2, l2));
                }
                if (near || (!BIAS && d00 < 31) || (p.window > 0 && d00 + 63 >= p.window)) {
                    const int n0 = d00 - (lane >> 2) + 2 * c0 - 24;
                    const float *bt = bias_row + g * bias_step;
                    auto entry = [&](int n) -> float {
                        float x = 0.f;
                        if (near)
                            x = bt[n];  // (-inf before distance 0)
                        else if (!BIAS && n < 0)
                            x = -INFINITY;
                        return p.window > 0 && n >= p.window ? -INFINITY : x;
                    };
#pragma unroll
                    for (int x = 0; x < 11; ++x) {  // b - a + 3
                        const uint64_t x2 = f2_pack(entry(n0 + 8 * x), entry(n0 + 8 * x + 1));
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            const int b = a + x - 3;
                            if (b >= 0 && b < 8) set_pair(w, a, b, f2_add(block_pair(w, a, b), x2));
                        }
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {  // pair 2 b + a % 2
                        float &e0 = w[half][2 * x], &e1 = w[half][2 * x + 1];
                        e0 = ex2_approx(e0);
                        e1 = ex2_approx(e1);
                        pk[x] = pack_bf16x2(e0, e1);
                    }
                    tmem_st_16x128b_x8(sc + static_cast<uint32_t>(half * 16 << 16), pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_PFULL));
                if (!wait_warp(bar(B_DPFULL), J & 1, c.abort_flag, p.err, kTimeoutNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float *dl = stat(st) + 128 + 64 * wg + 2 * c0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float d[32];
                    tmem_ld_16x256b_x8(dp + static_cast<uint32_t>(half * 16 << 16), d);
                    tmem_wait_ld_regs(d);
                    uint32_t pk[16];
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        const uint64_t l2 = *reinterpret_cast<const uint64_t *>(dl + 8 * b);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float *x = &d[4 * b + 2 * u];
                            f2_unpack(f2_mul(block_pair(w, 2 * half + u, b), f2_add(f2_pack(x[0], x[1]), l2)), x[0], x[1]);
                            pk[2 * b + u] = pack_bf16x2(x[0], x[1]);
                        }
                    }
                    tmem_st_16x128b_x8(dp + static_cast<uint32_t>(half * 16 << 16), pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_DSFULL));
                if (++q == t.n) {
                    q = 0;
                    ++g;
                }
            }
            if (BIAS && ok) {
                __syncwarp();
                if (table_here && lane == 0) mbar_arrive(bar(B_TABFREE + (items & 1)));
            }
            ok = ok && wait_warp(bar(B_DONE), items & 1, c.abort_flag, p.err, kTimeoutNs);
            if (!ok) break;
            tc_fence_after();
            const int64_t stride = wg ? p.dk_stride : p.dv_stride;
            __nv_bfloat16 *dst = (wg ? dk : dv) + static_cast<int64_t>(row) * stride;
            const bool v8 = aligned32(wg ? p.dk : p.dv, stride);
            const float f = wg ? p.scale : 1.f;
            const uint32_t acc = c.tmem + t_lane + (wg ? kDk : kDv);
            if (t.parts == 1) {
#pragma unroll 1
                for (int cc = 0; cc < HD / 32; ++cc) store_chunk(acc + cc * 32, f, dst + cc * 32, row < rows, v8);
            } else {
                const int slot = t.slot + kvh * t.parts;
                auto sums = [&](int part, int c4) -> float4 * {
                    return reinterpret_cast<float4 *>(p.split) + (static_cast<int64_t>(2 * (slot + part) + wg) * (HD / 4) + c4) * 128 + row;
                };
#pragma unroll 1
                for (int cc = 0; cc < HD / 32; ++cc) {
                    float o[32];
                    tmem_ld_32x32b_x32(acc + cc * 32, o);
                    tmem_wait_ld_regs(o);
#pragma unroll
                    for (int x = 0; x < 8; ++x) *sums(t.part, 8 * cc + x) = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                }
                // The last of the parts' warps w has all of their sums of its rows.
                __threadfence();
                __syncwarp();
                int before = 0;
                if (lane == 0) before = atomicAdd(p.arrived + 8 * slot + warp, 1);
                before = __shfl_sync(0xffffffffu, before, 0);
                if (before == t.parts - 1) {
                    __threadfence();
#pragma unroll 1
                    for (int c4 = 0; c4 < HD / 4; c4 += 4) {
                        float4 o[4] = {};
#pragma unroll 4
                        for (int part = 0; part < t.parts; ++part) {
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float4 s = __ldcg(sums(part, c4 + x));
                                o[x].x += s.x, o[x].y += s.y, o[x].z += s.z, o[x].w += s.w;
                            }
                        }
                        if (row < rows) {
                            uint4 *d4 = reinterpret_cast<uint4 *>(dst + 4 * c4);
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                d4[x] = make_uint4(pack_bf16x2(o[2 * x].x * f, o[2 * x].y * f), pack_bf16x2(o[2 * x].z * f, o[2 * x].w * f),
                                                   pack_bf16x2(o[2 * x + 1].x * f, o[2 * x + 1].y * f),
                                                   pack_bf16x2(o[2 * x + 1].z * f, o[2 * x + 1].w * f));
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_ACCFREE));
            ++items;
        }
    }
    teardown(c);
}

// ---------------------------------------------------------------------- dbias ---
// Sums the query tiles' partial sums, eight warps' for each, always in the same order: a block takes
// eight buckets of a head (a sector of a row), 128 threads a bucket.  4.5 us for 145 tiles of 32 heads, 32
// buckets (4.8 MB): latency.
constexpr int kBiasBuckets = 8;
__global__ void __launch_bounds__(1024)
    grad_bias_kernel(float *__restrict__ dbias, const float *__restrict__ partial, const int *__restrict__ counts, int num_heads,
                     int num_buckets) {
    __shared__ float s[32][kBiasBuckets];
    const int h = blockIdx.x, b = blockIdx.y * kBiasBuckets + threadIdx.x % kBiasBuckets;
    const int rows = *counts * 8;
    float t = 0.f;
    if (b < num_buckets) {
#pragma unroll 4
        for (int r = threadIdx.x / kBiasBuckets; r < rows; r += 1024 / kBiasBuckets)
            t += partial[((static_cast<int64_t>(r >> 3) * num_heads + h) * 8 + (r & 7)) * num_buckets + b];
    }
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    if ((threadIdx.x & 31) < kBiasBuckets) s[threadIdx.x >> 5][threadIdx.x & 31] = t;
    __syncthreads();
    if (threadIdx.x < kBiasBuckets && b < num_buckets) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
        dbias[b * num_heads + h] = t;
    }
}

// ------------------------------------------------------------------ host side ---
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Most tiles that sequences of `total` rows in all can have.
int64_t most_tiles(int total, int num_seqs) { return static_cast<int64_t>(total) / BM + num_seqs; }

// Places for the sums of split key tiles: tiles of fewer steps than kMinSteps have none, others less than a
// quarter of their steps.
int split_slots(int total_q, int total_k, int num_seqs, int num_heads) {
    const double steps = static_cast<double>(most_tiles(total_q, num_seqs)) * most_tiles(total_k, num_seqs) * num_heads;
    return steps / 4 < kMaxSlots ? static_cast<int>(steps / 4) : kMaxSlots;
}

// The workspace: lse2, delta, counts, lists, partial sums of dbias, sums of split key tiles (for 128 dims) and
// their counters, which of dQ's items are done again.
struct Workspace {
    int slots;
    size_t stat, q_list, k_list, partial, split, arrived, again;
    size_t bytes() const { return 2 * stat + 256 + q_list + k_list + partial + split + arrived + again; }
    Workspace(int total_q, int total_k, int num_seqs, int num_heads, int num_buckets)
        : slots(split_slots(total_q, total_k, num_seqs, num_heads)),
          stat(up256(static_cast<size_t>(total_q) * num_heads * sizeof(float))),
          q_list(up256(most_tiles(total_q, num_seqs) * sizeof(QTile))),
          k_list(up256((most_tiles(total_k, num_seqs) + slots) * sizeof(KTile))),
          partial(up256(static_cast<size_t>(most_tiles(total_q, num_seqs)) * num_heads * 8 * num_buckets * sizeof(float))),
          split(static_cast<size_t>(slots) * 2 * BM * 128 * sizeof(float)),
          arrived(up256(static_cast<size_t>(slots) * 8 * sizeof(int))),
          again(up256(static_cast<size_t>(most_tiles(total_q, num_seqs)) * num_heads * 4)) {}
};

template <class Kernel>
cudaError_t launch_tiles(Kernel kern, uint32_t smem, std::atomic<uint64_t> &set, int64_t items, const GradParams &p,
                         cudaStream_t stream) {
    if (items <= 0) return cudaSuccess;
    const cudaError_t e = smem_limit_once(kern, static_cast<int>(smem), set);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    kern<<<static_cast<unsigned>(items < sms ? items : sms), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int HD, bool BIAS>
cudaError_t launch_backward_d(GradParams &p, const PlanParams &plan, const PackedGradArgs &g, cudaStream_t stream) {
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
    const int table_blocks = BIAS ? (bias_stride(a.bias.last()) + 255) / 256 : 0;
    const dim3 grid((a.total_q + 7) / 8 + 1 + table_blocks, (a.num_heads + 7) / 8);
    grad_stat_kernel<HD><<<grid, 256, 0, stream>>>(static_cast<const uint4 *>(g.out), static_cast<const uint4 *>(g.dout), g.lse,
                                                   const_cast<float *>(p.lse2), p.delta, a.total_q, a.num_heads, plan,
                                                   const_cast<float *>(a.bias_table), a.bias, table_blocks);
    cudaError_t e = cudaGetLastError();
    static std::atomic<uint64_t> set[2];
    const int64_t q_items = a.total_q > 0 ? most_tiles(a.total_q, a.num_seqs) * a.num_heads : 0;
    const int64_t k_items = a.total_k > 0 ? (most_tiles(a.total_k, a.num_seqs) + plan.slots) * a.num_kv_heads : 0;
    if (e == cudaSuccess) e = launch_tiles(grad_q_kernel<HD, BIAS>, LayoutQ<HD, BIAS>::SMEM, set[0], q_items, p, stream);
    if (e == cudaSuccess) e = launch_tiles(grad_kv_kernel<HD, BIAS>, LayoutKv<HD, BIAS>::SMEM, set[1], k_items, p, stream);
    if (BIAS && e == cudaSuccess) {
        const dim3 blocks(a.num_heads, (a.bias.num_buckets + kBiasBuckets - 1) / kBiasBuckets);
        grad_bias_kernel<<<blocks, 1024, 0, stream>>>(g.dbias, p.partial, p.counts, a.num_heads, a.bias.num_buckets);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

bool packed_grad_workspace(int total_q, int total_k, int num_seqs, int num_heads, int num_buckets, size_t *bytes) {
    if (most_tiles(total_q, num_seqs) * num_heads > INT_MAX || most_tiles(total_k, num_seqs) * num_heads > INT_MAX) return false;
    *bytes = Workspace(total_q, total_k, num_seqs, num_heads, num_buckets).bytes();
    return true;
}

cudaError_t launch_packed_attn_backward(const PackedGradArgs &g, cudaStream_t stream) {
    const PackedArgs &a = g.fwd;
    GradParams p;
    memset(&p, 0, sizeof p);
    p.dq = static_cast<__nv_bfloat16 *>(g.dq);
    p.dk = static_cast<__nv_bfloat16 *>(g.dk);
    p.dv = static_cast<__nv_bfloat16 *>(g.dv);
    p.dq_stride = g.dq_stride;
    p.dk_stride = g.dk_stride;
    p.dv_stride = g.dv_stride;
    const Workspace w(a.total_q, a.total_k, a.num_seqs, a.num_heads, a.bias.num_buckets);
    uint8_t *at = static_cast<uint8_t *>(g.workspace);
    auto take = [&](size_t bytes) {
        uint8_t *const here = at;
        at += bytes;
        return here;
    };
    p.lse2 = reinterpret_cast<const float *>(take(w.stat));
    p.delta = reinterpret_cast<float *>(take(w.stat));
    PlanParams plan;
    plan.cu_q = a.cu_seqlens_q;
    plan.cu_k = a.cu_seqlens_k;
    plan.num_seqs = a.num_seqs;
    plan.total_q = a.total_q;
    plan.total_k = a.total_k;
    plan.max_q = a.max_seqlen_q;
    plan.max_k = a.max_seqlen_k;
    plan.window = a.sliding_window;
    plan.most[0] = static_cast<int>(most_tiles(a.total_q, a.num_seqs));
    plan.most[1] = static_cast<int>(most_tiles(a.total_k, a.num_seqs));
    plan.num_kv_heads = a.num_kv_heads;
    plan.group = a.num_heads / a.num_kv_heads;
    plan.slots = w.slots;
    plan.counts = reinterpret_cast<int *>(take(256));
    plan.q_list = reinterpret_cast<QTile *>(take(w.q_list));
    plan.k_list = reinterpret_cast<KTile *>(take(w.k_list));
    plan.err = a.err;
    p.counts = plan.counts;
    p.q_list = plan.q_list;
    p.k_list = plan.k_list;
    p.partial = reinterpret_cast<float *>(take(w.partial));
    p.split = reinterpret_cast<float *>(take(w.split));
    p.arrived = plan.arrived = reinterpret_cast<int *>(take(w.arrived));
    p.again = take(w.again);
    p.bias_table = a.bias_table;
    p.total_q = a.total_q;
    p.total_k = a.total_k;
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
        case 64: return bias ? launch_backward_d<64, true>(p, plan, g, stream) : launch_backward_d<64, false>(p, plan, g, stream);
        case 128: return bias ? launch_backward_d<128, true>(p, plan, g, stream) : launch_backward_d<128, false>(p, plan, g, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
