// decode_fp4.cu - decode over the 4-bit paged KV cache (fp4.cuh).
//
// For sequence b with L keys and query head h: out[b][h] = softmax(scale * q K^T) V over keys
// [max(0, L - w), L), K and V elements code * scale * kv_scale, read through block_table.
//
// A byte of cache holds 1.8 elements, so the kernel has to spend few instructions on each
// byte and keep the stream going without a pause:
//  * The keys of all (sequence, kv head, 16-head tile) segments are one flat list of 32-key
//    units, cut into equal ranges, one for each resident warp.  A warp streams its range
//    through its own ring of shared-memory stages without stopping at segment ends, so there
//    are no waves of blocks, no ragged tail and one pipeline fill a warp.
//  * 16 tokens of one kv head are 9 D contiguous bytes (rows of codes and scales), so a unit is
//    four runs (K and V of two 16-key halves) that the lanes copy 16 bytes at a time
//    (cp.async), a lane's chunks at constant distances.  (Bulk copies, which one lane issues,
//    took more issue slots: their operands go through uniform registers one copy at a time.)
//  * The products are f16 warp MMAs (m16n8k16, fp32 accumulate) with 16 keys as the M rows of
//    S^T = K Q^T and the head dims as those of O^T += V^T P^T, the query heads the 8 columns
//    of an n-tile (two n-tiles above 8 heads a kv head).  Codes become f16 by one conversion
//    for two and are scaled by one f16x2 product, exactly (fp4.cuh).  The softmax denominator
//    is one more MMA, with a matrix of ones in V's place.
//  * The MMA's key and dim indices are permuted so that a lane needs whole runs of a row: K
//    lane t of a quad takes dims D / 4 t .. of its key rows; V lane group g owns D / 8
//    consecutive dims (one scale a key) of keys 4 t .. 4 t + 3.  Loads are 8 bytes wide and, with
//    72-byte rows, free of bank conflicts for V; and a lane ends up with consecutive dims of
//    O for its heads, which it writes as whole vectors.
//  * A segment inside one warp's range is finished there.  A cut one leaves (m, l, O) of each
//    piece in the workspace and decode_fp4_combine_kernel (a programmatic dependent, which may
//    start as soon as the split kernel's inputs are complete) merges them.  When no sequence can be longer than kWholeUnits units, ranges are whole segments
//    and no combine is launched.
//
// Measured: 8 sequences of 81920 keys, 40/8 heads, 129 us a call (755 MB, 5.8 TB/s); 64 of
// 2304, 32/8 heads, 38 us (170 MB; 5 us to the first data, 3 of ragged ends, 3 of merge); 4 of
// 17-100, 8/2 heads of 64, 4.2 us (replayed from a graph).  Storing the new tokens as well takes 1 to 2 us
// more with short sequences (40.7 us against 38.8, 64 of 512-4096), nothing with long ones.  Without its arithmetic the long call takes 117 us: the loads and
// the issue of 594 instructions a unit (128 conversions at half rate among them) bound it
// together.

#include <atomic>

#include "decode_common.cuh"
#include "fp4.cuh"
#include "pa_common.cuh"
#include "pa_internal.h"
#include "sm100_ptx.cuh"

namespace pa {

namespace {

using namespace sm100;

// Independent warps of a block, one block an SM: 168 registers a thread with one n-tile of heads
// (12 warps), 255 with two (8 warps).  (As three blocks of four warps an SM the same kernel took 133
// us for 128.5, 8 x 81920 keys, 40/8 heads: the schedulers prefer an older block's warps, so of
// equal ranges the last block's ended at 121 us where the first one's did at 93, and ran alone
// at the end; the warps of one block end together.)
__host__ __device__ constexpr int warps_of(int nt) { return nt == 1 ? 12 : 8; }
constexpr int kScan = 128;         // threads that add up the sequences' units
constexpr int kUnit = 32;          // keys of a unit: two 16-key halves
constexpr int kStages = 3;         // ring stages of a warp, one unit of K and V each
constexpr int kMinUnits = 4;       // smallest range of a warp (128 keys)
constexpr int kWholeUnits = 5;     // spans up to this many units are never cut
constexpr int kMergeWarps = 8;     // warps of a combine block

struct Params {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const int32_t *block_table;
    int max_num_blocks;
    const int32_t *seq_lens;
    int batch;
    int64_t seq_cap;
    int64_t num_blocks;
    int log2_bs;
    int num_heads;
    int num_kv_heads;
    int group;
    int head_tiles;
    int window;
    float scale_log2;  // scale * kv_scale * log2(e)
    float kv_scale;
    int workers;       // warps of the grid
    int whole_units;   // > 0: ranges are whole segments of at most this many units
    float *pieces;     // [workers][2][tile heads][D + 2]: O, m, l of a cut segment's piece
    int tile_heads;    // min(group, 16)
    // Fused store of each sequence's new token (null when not fused).
    const __nv_bfloat16 *key;
    const __nv_bfloat16 *value;
    const int32_t *slot_mapping;
    uint8_t *k_cache_w;
    uint8_t *v_cache_w;
    // Varlen layout: only sequences with one query row, at row q_rows[b] (null: row b).
    const int32_t *q_rows;
    int total_q;
    int check_rows;
    int max_seqlen_q;
    const int32_t *cu_k;
    int after_prefill;
    unsigned *err;
};

// Units of sequence b and its key range: 0 without keys, -1 for a sequence that is not decoded here.
// EARLY: read by a kernel that has not waited for what precedes it (the merge), from the L2, where
// the writes that the split kernel waited for are.
template <bool EARLY = false>
__device__ __forceinline__ int seq_units(const Params &p, int b, SeqRange &r, bool report) {
    auto load = [](const int32_t *at) { return EARLY ? __ldcg(at) : *at; };
    if (p.q_rows != nullptr) {
        const int r0 = load(p.q_rows + b);
        const int sq = load(p.q_rows + b + 1) - r0;
        if (report && p.check_rows) {
            const int sk = load(p.seq_lens + b);
            if (sq < 0 || sq > p.max_seqlen_q || sq > sk) flag_error(p.err, kErrQueryLen);
            if (p.cu_k != nullptr && p.cu_k[b + 1] - p.cu_k[b] != sk) flag_error(p.err, kErrSeqlensK);
        }
        if (sq != 1 || r0 < 0 || r0 >= p.total_q) {
            if (report && sq == 1) flag_error(p.err, kErrQueryLen);
            r.L = r.start = r.base = 0;
            return -1;
        }
    }
    r = decode_range(load(p.seq_lens + b), p.seq_cap, p.window, 0, p.err, report);
    return (r.L - r.base + kUnit - 1) / kUnit;
}

// Units of a worker's range when the whole list has `total`.
__device__ __forceinline__ long long range_of(const Params &p, long long total) {
    const long long r = (total + p.workers - 1) / p.workers;
    return r < kMinUnits ? kMinUnits : r;
}

// Shared-memory loads at a constant offset from a register address.
template <int OFF>
__device__ __forceinline__ void lds_64(uint32_t addr, uint32_t &a, uint32_t &b) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2 + %3];" : "=r"(a), "=r"(b) : "r"(addr), "n"(OFF));
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(v) : "r"(addr), "n"(OFF));
    return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v) : "r"(addr), "n"(OFF));
    return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(v) : "r"(addr), "n"(OFF));
    return v;
}

// D(16x8 f32) = A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                   uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The codes (D / 32 words, two k-steps each) and scales (as f16x2) of a lane's part of a K row, at
// byte OFF from the lane's addresses in a 16-key half.
template <int D, int OFF>
__device__ __forceinline__ uint32_t k_row(uint32_t codes, uint32_t scales, uint32_t (&w)[D / 32]) {
    if constexpr (D == 128) {  // 72-byte rows: 8-byte aligned
        lds_64<OFF>(codes, w[0], w[1]);
        lds_64<OFF + 8>(codes, w[2], w[3]);
        return fp4::e4m3x2_to_f16x2(lds_u16<OFF>(scales));
    } else {  // 36-byte rows: 4-byte aligned
        w[0] = lds_32<OFF>(codes);
        w[1] = lds_32<OFF + 4>(codes);
        return fp4::e4m3x2_to_f16x2(lds_u8<OFF>(scales));
    }
}

// V codes of one key row: the lane's D / 8 dims.
template <int D, int OFF>
__device__ __forceinline__ void v_row(uint32_t codes, uint32_t (&w)[D / 64]) {
    if constexpr (D == 128)
        lds_64<OFF>(codes, w[0], w[1]);
    else
        w[0] = lds_32<OFF>(codes);
}

__device__ __forceinline__ void sts_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// One (sequence, kv head, head tile): where its keys and query rows are.
struct Segment {
    int b;
    int kvh;
    int ht;
    SeqRange r;
    int units;
};

// The next segment of the list (the caller knows that there is one).
__device__ __forceinline__ void advance(const Params &p, Segment &s) {
    if (++s.ht < p.head_tiles) return;
    s.ht = 0;
    if (++s.kvh < p.num_kv_heads) return;
    s.kvh = 0;
    do {
        ++s.b;
        s.units = max(seq_units(p, s.b, s.r, false), 0);
    } while (s.units == 0);
}

// Where a warp's copies are: ahead of its products.
struct Ahead {
    Segment seg;
    int unit;  // next unit of the segment
    int left;  // units of the warp's range not listed yet
};

template <int D, int NT>
__device__ __forceinline__ void split_body(const Params &p) {
    constexpr int RB = fp4::row_bytes(D);
    constexpr int HB = 16 * RB;         // bytes of a 16-key half of K (or V)
    constexpr int SB = 4 * HB;          // bytes of a stage: K and V of half 0, then of half 1
    constexpr int KSTEPS = D / 16;
    constexpr int VW = D / 64;          // words of V codes a lane takes of a key row
    constexpr int VD = 8 * VW;          // dims of V a lane owns
    constexpr int MT = D / 16;          // m-tiles of O^T

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Ahead s_ahead[warps_of(NT)];
    __shared__ long long part_sum[kScan];
    __shared__ long long s_total;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int HT = p.num_kv_heads * p.head_tiles;  // segments of a sequence
    constexpr int kWarps = warps_of(NT);
    const uint32_t ring = smem_u32(smem) + warp * kStages * SB;
    const uint64_t policy = l2_policy_evict_first();

    // ---- this warp's range [f, f_end) of the flat unit list ----
    // Worker v * blocks + c is warp v of block c: few workers spread over many SMs.
    const int w = warp * gridDim.x + blockIdx.x;
    const int chunk = (p.batch + kScan - 1) / kScan;
    const bool report = blockIdx.x == 0;
    if (threadIdx.x < kScan) {
        long long sum = 0;
        const int b0 = threadIdx.x * chunk, b1 = min(p.batch, b0 + chunk);
        if (p.whole_units == 0 || report)
            for (int b = b0; b < b1; ++b) {
                SeqRange r;
                sum += max(seq_units(p, b, r, report), 0);
            }
        part_sum[threadIdx.x] = sum;
    }
    __syncthreads();
    if (warp == 0) {
        // Exclusive prefix of the 128 partial sums, four to a lane.
        long long v[4], run = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = run;
            run += part_sum[4 * lane + i];
        }
        long long inc = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) part_sum[4 * lane + i] = inc - run + v[i];
        if (lane == 31) s_total = inc;
    }
    __syncthreads();

    long long f, f_end;       // flat range
    Segment seg;              // segment at f
    int unit = 0;             // f's unit in it
    const int n_seg = p.batch * HT;
    if (p.whole_units > 0) {
        // Whole segments: segment w of the list, at most one a worker (the grid covers them).
        f = w;
        f_end = min(w + 1, n_seg);
        seg.b = w / HT;
    } else {
        const long long total = s_total * HT;
        const long long range = range_of(p, total);
        f = min(total, range * w);
        f_end = min(total, f + range);
    }
    if (f < f_end) {
        // The sequence that holds unit f: the thread chunk, then the sequence inside it.
        if (p.whole_units == 0) {
            const long long sf = f / HT;  // f lies in the sequence that holds sequence-unit sf
            int c = 0;
#pragma unroll
            for (int step = 64; step > 0; step >>= 1)
                if (part_sum[c + step] <= sf) c += step;
            long long begin = part_sum[c];
            int b = c * chunk;
            for (;; ++b) {
                SeqRange r;
                const int u = max(seq_units(p, b, r, false), 0);
                if (sf < begin + u) {
                    seg.b = b;
                    seg.r = r;
                    seg.units = u;
                    break;
                }
                begin += u;
            }
            const long long in_seq = f - begin * HT;
            const int h = static_cast<int>(in_seq / seg.units);
            unit = static_cast<int>(in_seq - static_cast<long long>(h) * seg.units);
            seg.kvh = h / p.head_tiles;
            seg.ht = h - seg.kvh * p.head_tiles;
        } else {
            const int h = w - seg.b * HT;
            seg.kvh = h / p.head_tiles;
            seg.ht = h - seg.kvh * p.head_tiles;
            seg.units = max(seq_units(p, seg.b, seg.r, false), 0);
            f_end = f + seg.units;
        }
    }
    int todo = f < f_end ? static_cast<int>(f_end - f) : 0;  // units this warp has to read

    // ---- rows without keys (zeros), and their new tokens ----
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        SeqRange r;
        if (seq_units(p, b, r, false) != 0) continue;
        const int64_t row = p.q_rows != nullptr ? p.q_rows[b] : b;
        for (int i = threadIdx.x; i < p.num_heads * D / 2; i += kWarps * 32)
            reinterpret_cast<uint32_t *>(p.out + row * p.num_heads * D)[i] = 0u;
        if (p.slot_mapping != nullptr && p.slot_mapping[b] >= 0) {
            // No position of the sequence owns the slot; the row is written all the same.
            const int64_t slot = p.slot_mapping[b];
            if (threadIdx.x == 0)
                flag_error(p.err, slot < (p.num_blocks << p.log2_bs) ? kErrSlotMismatch : kErrSlotRange);
            if (slot < (p.num_blocks << p.log2_bs)) {
                const int bs_mask = (1 << p.log2_bs) - 1;
                for (int i = threadIdx.x; i < p.num_kv_heads * 2 * (D / 16); i += kWarps * 32) {
                    const int gr = i % (D / 16);
                    const int which = i / (D / 16) & 1;
                    const int h = i / (2 * (D / 16));
                    const __nv_bfloat16 *src = (which ? p.value : p.key) +
                                               (static_cast<int64_t>(b) * p.num_kv_heads + h) * D + 16 * gr;
                    uint32_t x[8], sc;
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = reinterpret_cast<const uint32_t *>(src)[k];
                    const uint2 c = fp4::quant_group(x, p.kv_scale, 6.f * p.kv_scale, sc);
                    uint8_t *dst = (which ? p.v_cache_w : p.k_cache_w) +
                                   ((((slot >> p.log2_bs) * p.num_kv_heads + h) << p.log2_bs) +
                                    (slot & bs_mask)) * RB;
                    reinterpret_cast<uint32_t *>(dst)[2 * gr] = c.x;
                    reinterpret_cast<uint32_t *>(dst)[2 * gr + 1] = c.y;
                    dst[D / 2 + gr] = static_cast<uint8_t>(sc);
                }
            }
        }
    }
    if (todo == 0) return;

    // Q^T fragments of a segment: the B operand of S^T.  k-step ks is dims D / 4 t + 4 ks .. + 3;
    // head 8 j + g.  Heads past the group are zero.
    uint32_t qf[NT][KSTEPS][2];
    auto load_q = [&]() {
        const int rows_valid = min(16, p.group - seg.ht * 16);
        const int64_t row = p.q_rows != nullptr ? p.q_rows[seg.b] : seg.b;
        const __nv_bfloat16 *qb = p.q + (row * p.num_heads + seg.kvh * p.group + seg.ht * 16) * D;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < KSTEPS / 2; ++c) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (8 * j + g < rows_valid)
                    x = reinterpret_cast<const uint4 *>(qb + (8 * j + g) * D + D / 4 * t)[c];
                qf[j][2 * c][0] = bf16x2_to_f16x2(x.x);
                qf[j][2 * c][1] = bf16x2_to_f16x2(x.y);
                qf[j][2 * c + 1][0] = bf16x2_to_f16x2(x.z);
                qf[j][2 * c + 1][1] = bf16x2_to_f16x2(x.w);
            }
    };
    load_q();  // in flight beside the block table

    // ---- the issue side: units ahead of the consumer, across segments ----
    // Its place is kept in shared memory: it is needed once for 16 units.  In registers are the
    // byte offsets of the next units' halves, lane i that of half i (odd: past the sequence or
    // a bad table entry, read as zeros), and how many units they cover.
    s_ahead[warp].seg = seg;
    s_ahead[warp].unit = unit;
    s_ahead[warp].left = todo;
    __syncwarp();
    const int64_t block_bytes = (static_cast<int64_t>(p.num_kv_heads) << p.log2_bs) * RB;
    const int bs_mask = (1 << p.log2_bs) - 1;
    long long half_off = 0;
    int listed = 0, next = 0;  // units of the list, units issued of it
    auto list_units = [&]() {
        Ahead a = s_ahead[warp];
        next = listed = 0;
        if (a.left == 0) return;
        if (a.unit == a.seg.units) {
            advance(p, a.seg);
            a.unit = 0;
        }
        listed = min(16, min(a.left, a.seg.units - a.unit));
        const int key = a.seg.r.base + kUnit * a.unit + 16 * lane;
        half_off = 1;
        if (lane < 2 * listed && key < a.seg.r.L) {
            const int blk = p.block_table[static_cast<int64_t>(a.seg.b) * p.max_num_blocks + (key >> p.log2_bs)];
            if (blk >= 0 && blk < p.num_blocks) {
                half_off += blk * block_bytes + ((a.seg.kvh << p.log2_bs) + (key & bs_mask)) * RB - 1;
            } else {
                flag_error(p.err, kErrBlockRange);
            }
        }
        a.unit += listed;
        a.left -= listed;
        __syncwarp();
        if (lane == 0) s_ahead[warp] = a;
        __syncwarp();
    };
    // Issue the next unit (if there is one) into stage st.  Of each run's CH 16-byte chunks (K and V
    // of half 0, K and V of half 1), whole sets of 32 are a copy of the warp each; the rests of
    // the four runs share one, CT lanes for a run.
    constexpr int CH = HB / 16, CT = CH % 32;
    static_assert(4 * CT <= 32, "the rests of the four runs fit one copy");
    const int t_run = lane / CT;  // (4 and above: no part in the last copy)
    const uint32_t t_at = (CH - CT + lane % CT) * 16;
    const uint8_t *k_lane = p.k_cache + 16 * lane, *v_lane = p.v_cache + 16 * lane;
    const uint8_t *t_lane = ((t_run & 1) ? p.v_cache : p.k_cache) + t_at;
    const uint32_t t_dst = ring + t_run * HB + t_at;
    auto issue = [&](int st) {
        if (next == listed) list_units();
        if (next < listed) {
            const uint32_t dst = ring + st * SB + 16 * lane;
            long long off[2];
            uint32_t size[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                off[h] = __shfl_sync(0xffffffffu, half_off, 2 * next + h);
                size[h] = (off[h] & 1) ? 0u : 16u;
                off[h] &= ~1ll;
#pragma unroll
                for (int i = 0; i < CH / 32; ++i) {
                    cp_async_16_policy(dst + 2 * h * HB + 512 * i, k_lane + off[h] + 512 * i, size[h], policy);
                    cp_async_16_policy(dst + (2 * h + 1) * HB + 512 * i, v_lane + off[h] + 512 * i, size[h], policy);
                }
            }
            if (t_run < 4)
                cp_async_16_policy(t_dst + st * SB, t_lane + (t_run < 2 ? off[0] : off[1]), t_run < 2 ? size[0] : size[1], policy);
            ++next;
        }
        cp_async_commit();
    };
    // kStages - 1 units in flight before the first one is waited for; every step commits one
    // group, so that counting groups counts units.
#pragma unroll 1
    for (int s = 0; s < kStages - 1; ++s) issue(s);

    // ---- the consumer side ----
    // O^T accumulators: tile i of 16 rows: row g is dim VD g + 2 i, row g + 8 dim VD g + 2 i + 1;
    // columns (heads) 8 j + 2 t and + 1.
    float o[NT][MT][4];
    // Per head: m_run is the reference maximum the weights are taken against (base 2); it moves
    // only when a score exceeds it by more than 8.  lsum is the tile of the ones' product: every
    // row of it is the denominator.
    float m_run[NT][2], lsum[NT][4];
    auto reset = [&]() {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int i = 0; i < MT; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
            lsum[j][0] = lsum[j][1] = lsum[j][2] = lsum[j][3] = 0.f;
            m_run[j][0] = m_run[j][1] = -INFINITY;
        }
    };
    reset();
    int first_unit = unit;  // first unit of the segment's piece in this range

    // MMA row r of a unit is key 4 (r % 8 / 2) + r % 2 + 2 (r / 8): rows 2 t, 2 t + 1, 2 t + 8 and
    // 2 t + 9 are keys 4 t .. 4 t + 3.
    const int key_a = 4 * (g >> 1) + (g & 1);  // of row g; row g + 8 is key_a + 2
    const uint32_t k_off = key_a * RB + D / 8 * t, ks_off = key_a * RB + D / 2 + (D == 128 ? 2 * t : t);
    const uint32_t v_off = 4 * t * RB + 4 * VW * g, vs_off = 4 * t * RB + D / 2 + (D == 128 ? g : g >> 1);
    constexpr uint32_t kOnes[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};

    int st = 0;
#pragma unroll 1
    for (;;) {
        // The stage that the previous unit left takes the next one.
        issue(st == 0 ? kStages - 1 : st - 1);
        cp_async_wait<kStages - 1>();
        __syncwarp();
        const uint32_t kb = ring + st * SB;
        const uint32_t vb = kb + HB;  // of half 0; half 1 is 2 HB further
        const int key0 = seg.r.base + kUnit * unit;
        const bool last_unit = unit == seg.units - 1;

        // The new token's rows replace the unit's last key in shared memory, and are written
        // to the cache: this unit's copy may or may not have seen that write.
        if (last_unit && p.slot_mapping != nullptr) {
            const int slot = p.slot_mapping[seg.b];
            const int pos = seg.r.L - 1;
            const int64_t num_slots = p.num_blocks << p.log2_bs;
            if (slot >= num_slots) {
                if (lane == 0) flag_error(p.err, kErrSlotRange);
            } else if (slot >= 0) {
                const int blk = p.block_table[static_cast<int64_t>(seg.b) * p.max_num_blocks + (pos >> p.log2_bs)];
                const bool match = ((static_cast<int64_t>(blk) << p.log2_bs) | (pos & bs_mask)) == slot;
                if (!match && lane == 0) flag_error(p.err, kErrSlotMismatch);
                if (lane < 2 * (D / 16)) {
                    const int which = lane / (D / 16), gr = lane % (D / 16);
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(
                        (which ? p.value : p.key) +
                        (static_cast<int64_t>(seg.b) * p.num_kv_heads + seg.kvh) * D + 16 * gr);
                    uint32_t x[8], sc;
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = src[k];
                    const uint2 c = fp4::quant_group(x, p.kv_scale, 6.f * p.kv_scale, sc);
                    uint8_t *dst = (which ? p.v_cache_w : p.k_cache_w) +
                                   ((((static_cast<int64_t>(slot) >> p.log2_bs) * p.num_kv_heads + seg.kvh)
                                     << p.log2_bs) + (slot & bs_mask)) * RB;
                    reinterpret_cast<uint32_t *>(dst)[2 * gr] = c.x;
                    reinterpret_cast<uint32_t *>(dst)[2 * gr + 1] = c.y;
                    dst[D / 2 + gr] = static_cast<uint8_t>(sc);
                    if (match) {
                        const int j = pos - key0;
                        const uint32_t row = (which ? vb : kb) + (j >> 4) * 2 * HB + (j & 15) * RB;
                        sts_u32(row + 8 * gr, c.x);
                        sts_u32(row + 8 * gr + 4, c.y);
                        asm volatile("st.shared.u8 [%0], %1;" ::"r"(row + D / 2 + gr), "r"(sc) : "memory");
                    }
                }
                __syncwarp();
            }
        }

        // S^T = K Q^T of the two halves, in turn: a step of one covers the latency of the other's.
        float s[2][NT][4];
        uint32_t wa[2][D / 32], wb[2][D / 32], sca[2], scb[2];  // codes and scales of rows g and g + 8
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t ca = kb + 2 * h * HB + k_off, cs = kb + 2 * h * HB + ks_off;
            sca[h] = k_row<D, 0>(ca, cs, wa[h]);
            scb[h] = k_row<D, 2 * RB>(ca, cs, wb[h]);
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            const uint32_t pick = (x >> 1) ? 0x3232 : 0x1010;  // a scale for two words
            uint32_t fa[2][4], fb[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t sa = __byte_perm(sca[h], 0u, pick), sb = __byte_perm(scb[h], 0u, pick);
                fp4::e2m1x8_to_f16x2x4(wa[h][x], fa[h]);
                fp4::e2m1x8_to_f16x2x4(wb[h][x], fb[h]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    fa[h][k] = fp4::mul_f16x2(fa[h][k], sa);
                    fb[h][k] = fp4::mul_f16x2(fb[h][k], sb);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a[4] = {fa[h][2 * k], fb[h][2 * k], fa[h][2 * k + 1], fb[h][2 * k + 1]};
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (x == 0 && k == 0)
                            mma_f16_16816_zero(s[h][j], a, qf[j][0][0], qf[j][0][1]);
                        else
                            mma_f16_16816(s[h][j], a, qf[j][2 * x + k][0], qf[j][2 * x + k][1]);
                    }
                }
        }

        // V codes and scales of keys 4 t .. 4 t + 3 of each half.
        uint32_t vw[2][4][VW], vs[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t c = vb + 2 * h * HB + v_off, x = vb + 2 * h * HB + vs_off;
            v_row<D, 0>(c, vw[h][0]);
            v_row<D, RB>(c, vw[h][1]);
            v_row<D, 2 * RB>(c, vw[h][2]);
            v_row<D, 3 * RB>(c, vw[h][3]);
            vs[h][0] = lds_u8<0>(x);
            vs[h][1] = lds_u8<RB>(x);
            vs[h][2] = lds_u8<2 * RB>(x);
            vs[h][3] = lds_u8<3 * RB>(x);
        }

        // Mask (edge units only): element e of half h is key 16 h + key_a + (e & 2) and head
        // 2 t + (e & 1).  Rows outside the range may hold anything: a zero scale makes V zeros.
        if (key0 < seg.r.start || key0 + kUnit > seg.r.L) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + 16 * h + key_a + (e & 2);
                    if (key < seg.r.start || key >= seg.r.L)
#pragma unroll
                        for (int j = 0; j < NT; ++j) s[h][j][e] = -INFINITY;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = key0 + 16 * h + 4 * t + k;
                    if (key < seg.r.start || key >= seg.r.L) vs[h][k] = 0u;
                }
            }
        }
        // Online softmax per head column, the scale (> 0) folded into the exponent.
        float mx[NT][2];
        bool over = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[j][e] = fmaxf(max3f(s[0][j][e], s[0][j][e + 2], s[1][j][e]), s[1][j][e + 2]) * p.scale_log2;
                over |= mx[j][e] > m_run[j][e] + 8.f;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float fr[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = mx[j][e];
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    const bool nd = m > m_run[j][e] + 8.f;
                    fr[e] = nd ? ex2_approx(m_run[j][e] - m) : 1.f;
                    if (nd) m_run[j][e] = m;
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[j][i][0] *= fr[0];
                    o[j][i][1] *= fr[1];
                    o[j][i][2] *= fr[0];
                    o[j][i][3] *= fr[1];
                }
                lsum[j][0] *= fr[0];
                lsum[j][1] *= fr[1];
            }
        }
        // P^T (B operand): f16 weights packed per key row and transposed; the ones' product sums
        // the rounded weights that V's product uses.
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float m0 = m_run[j][0] == -INFINITY ? 0.f : m_run[j][0];
            const float m1 = m_run[j][1] == -INFINITY ? 0.f : m_run[j][1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float *x = s[h][j];
                pb[h][j][0] = movmatrix_trans(pack_f16x2(ex2_approx(fmaf(x[0], p.scale_log2, -m0)),
                                                         ex2_approx(fmaf(x[1], p.scale_log2, -m1))));
                pb[h][j][1] = movmatrix_trans(pack_f16x2(ex2_approx(fmaf(x[2], p.scale_log2, -m0)),
                                                         ex2_approx(fmaf(x[3], p.scale_log2, -m1))));
                mma_f16_16816(lsum[j], kOnes, pb[h][j][0], pb[h][j][1]);
            }
        }
        // O^T += V^T P^T: the codes of two keys and one dim meet in a byte, low code first.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t s01 = fp4::e4m3x2_to_f16x2(vs[h][0] | (vs[h][1] << 8));
            const uint32_t s23 = fp4::e4m3x2_to_f16x2(vs[h][2] | (vs[h][3] << 8));
#pragma unroll
            for (int x = 0; x < VW; ++x) {
                constexpr uint32_t LO = 0x0f0f0f0fu;
                const uint32_t k0 = vw[h][0][x], k1 = vw[h][1][x], k2 = vw[h][2][x], k3 = vw[h][3][x];
                uint32_t f0[4], f1[4], f2[4], f3[4];
                fp4::e2m1x8_to_f16x2x4((k0 & LO) | ((k1 << 4) & ~LO), f0);  // even dims
                fp4::e2m1x8_to_f16x2x4(((k0 >> 4) & LO) | (k1 & ~LO), f1);  // odd dims
                fp4::e2m1x8_to_f16x2x4((k2 & LO) | ((k3 << 4) & ~LO), f2);
                fp4::e2m1x8_to_f16x2x4(((k2 >> 4) & LO) | (k3 & ~LO), f3);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a[4] = {fp4::mul_f16x2(f0[k], s01), fp4::mul_f16x2(f1[k], s01),
                                           fp4::mul_f16x2(f2[k], s23), fp4::mul_f16x2(f3[k], s23)};
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma_f16_16816(o[j][4 * x + k], a, pb[h][j][0], pb[h][j][1]);
                }
            }
        }
        __syncwarp();
        if (++st == kStages) st = 0;
        --todo;
        ++unit;
        if (!last_unit && todo > 0) continue;

        // ---- end of the segment's piece: lanes t hold heads 2 t, 2 t + 1 of each n-tile ----
        const int rows_valid = min(16, p.group - seg.ht * 16);
        const bool whole = first_unit == 0 && last_unit;
        const int64_t row = p.q_rows != nullptr ? p.q_rows[seg.b] : seg.b;
        const int64_t h0 = row * p.num_heads + seg.kvh * p.group + seg.ht * 16;
        // A range starts inside at most one segment and ends inside at most one that began in it.
        float *piece = p.pieces + (static_cast<int64_t>(w) * 2 + (first_unit > 0 ? 0 : 1)) *
                                      p.tile_heads * (D + 2);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * j + 2 * t + e;
                if (h >= rows_valid) continue;
                if (whole) {
                    const float inv = p.kv_scale / lsum[j][e];
                    uint32_t x[MT];
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        x[i] = pack_bf16x2(o[j][i][e] * inv, o[j][i][e + 2] * inv);
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + (h0 + h) * D + VD * g);
#pragma unroll
                    for (int i = 0; i < MT / 4; ++i)
                        dst[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                } else {
                    float *ph = piece + h * (D + 2);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        *reinterpret_cast<float2 *>(ph + VD * g + 2 * i) =
                            make_float2(o[j][i][e], o[j][i][e + 2]);
                    if (g == 0) *reinterpret_cast<float2 *>(ph + D) = make_float2(m_run[j][e], lsum[j][e]);
                }
            }
        if (todo == 0) break;
        // Next segment.
        advance(p, seg);
        unit = first_unit = 0;
        load_q();
        reset();
    }
    cp_async_wait<0>();
}

template <int D, int NT>
__global__ void __launch_bounds__(warps_of(NT) * 32, 1)
    decode_fp4_split_kernel(const __grid_constant__ Params p) {
    // Always launched as a programmatic dependent, so that its launch overlaps the end of whatever
    // precedes it on the stream; beside a prefill (which itself began when all before it was
    // complete) it starts at once, else it waits here.  The merge reads the lengths before it waits
    // for this grid, so it is let in only behind this wait: what precedes the call may write them.
    // (For the same reason the inputs are read by ordinary loads: they may have been written while
    // this grid was there already, which read-only loads do not allow.)
    if (!p.after_prefill) griddep_wait();
    griddep_launch_dependents();
    split_body<D, NT>(p);
    // As a programmatic dependent of the prefill kernel of the same call, this grid (and what
    // waits for it) completes after the prefill: its last block waits for the prefill grid.
    if (p.after_prefill && blockIdx.x == gridDim.x - 1) griddep_wait();
}

// Merge of the pieces of the cut segments, a block taking consecutive (segment, head) items and
// as many warps as there are for an item sharing its pieces (one long sequence may be cut into a
// hundred).  With piece i holding (m_i, l_i, O_i):
//     M = max m_i,  out = kv_scale * sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// Where a segment is cut follows from the lengths alone, so that is worked out before the wait
// for the split grid (whose blocks have all passed theirs, so the lengths are the call's); after it
// there is one round trip for eight pieces.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) decode_fp4_combine_kernel(const __grid_constant__ Params p) {
    constexpr int PER = D / 32;
    constexpr int BATCH = 8;  // pieces in flight
    __shared__ long long sums[2][kMergeWarps];
    __shared__ float part[kMergeWarps][D + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int HT = p.num_kv_heads * p.head_tiles;
    const int64_t items = static_cast<int64_t>(p.batch) * HT * p.tile_heads;
    const int64_t per_block = (items + gridDim.x - 1) / gridDim.x;
    const int64_t i0 = blockIdx.x * per_block, i1 = min(items, i0 + per_block);
    int b = static_cast<int>(min(i0 / (HT * p.tile_heads), static_cast<int64_t>(p.batch)));
    SeqRange r;
    long long before = 0, total = 0;  // units of sequences before b, and of all
    for (int k = threadIdx.x; k < p.batch; k += kMergeWarps * 32) {
        const int u = max(seq_units<true>(p, k, r, false), 0);
        total += u;
        if (k < b) before += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane == 0) {
        sums[0][warp] = before;
        sums[1][warp] = total;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int v = 0; v < kMergeWarps; ++v) {
        before += sums[0][v];
        total += sums[1][v];
    }
    const long long range = range_of(p, total * HT);
    int units = b < p.batch ? max(seq_units<true>(p, b, r, false), 0) : 0;
    griddep_launch_dependents();
    int share = kMergeWarps;  // warps an item
    while (share > 1 && share * per_block > kMergeWarps) share >>= 1;
    const int per_round = kMergeWarps / share;
    const int sub = warp & (share - 1);
    griddep_wait();
    for (int64_t it = i0; it < i1; it += per_round) {
        const int64_t item = it + warp / share;
        const int64_t s = item / p.tile_heads;
        const int h = static_cast<int>(item - s * p.tile_heads);
        const int bi = item < i1 ? static_cast<int>(s / HT) : b;
        while (b < bi) {
            before += units;
            units = max(seq_units<true>(p, ++b, r, false), 0);
        }
        const int hs = static_cast<int>(s - static_cast<int64_t>(b) * HT);
        const int kvh = hs / p.head_tiles, ht = hs - kvh * p.head_tiles;
        const long long f0 = before * HT + static_cast<long long>(hs) * units;
        const bool valid = item < i1 && units > 0 && h < p.group - ht * 16;
        const int w0 = valid ? static_cast<int>(f0 / range) : 0;
        const int n = valid ? static_cast<int>((f0 + units - 1) / range) - w0 + 1 : 0;  // pieces
        float M = -INFINITY, den = 0.f, acc[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[k] = 0.f;
        if (n > 1) {
            // Piece 0 is the second one of its worker, which started the segment; the others are
            // the first ones of theirs.
            auto piece = [&](int i) {
                return p.pieces + (static_cast<int64_t>(w0 + i) * 2 + (i == 0 ? 1 : 0)) * p.tile_heads * (D + 2) +
                       h * (D + 2);
            };
            for (int k0 = sub; k0 < n; k0 += BATCH * share) {
                float2 v[BATCH][PER / 2], ml[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int i = k0 + k * share;
                    ml[k] = make_float2(-INFINITY, 0.f);
                    if (i < n) {
                        const float2 *src = reinterpret_cast<const float2 *>(piece(i));
                        ml[k] = src[D / 2];
#pragma unroll
                        for (int c = 0; c < PER / 2; ++c) v[k][c] = src[lane + 32 * c];
                    }
                }
                float m_new = M;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) m_new = fmaxf(m_new, ml[k].x);
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                const float f = ex2_approx(M - m_use);
                den *= f;
#pragma unroll
                for (int c = 0; c < PER; ++c) acc[c] *= f;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    if (k0 + k * share >= n) break;
                    const float wt = ex2_approx(ml[k].x - m_use);
                    den += wt * ml[k].y;
#pragma unroll
                    for (int c = 0; c < PER / 2; ++c) {
                        acc[2 * c] += wt * v[k][c].x;
                        acc[2 * c + 1] += wt * v[k][c].y;
                    }
                }
                M = m_new;
            }
        }
        if (share > 1) {
            __syncthreads();  // the previous round's sums have been read
#pragma unroll
            for (int c = 0; c < PER; ++c) part[warp][32 * c + lane] = acc[c];
            if (lane == 0) {
                part[warp][D] = M;
                part[warp][D + 1] = den;
            }
            __syncthreads();
            if (sub != 0 || n <= 1) continue;
            float m_all = M;
            for (int v = 1; v < share; ++v) m_all = fmaxf(m_all, part[warp + v][D]);
            const float m_use = m_all == -INFINITY ? 0.f : m_all;
            const float f0w = ex2_approx(M - m_use);
            den *= f0w;
#pragma unroll
            for (int c = 0; c < PER; ++c) acc[c] *= f0w;
            for (int v = 1; v < share; ++v) {
                const float f = ex2_approx(part[warp + v][D] - m_use);
                den += f * part[warp + v][D + 1];
#pragma unroll
                for (int c = 0; c < PER; ++c) acc[c] += f * part[warp + v][32 * c + lane];
            }
        }
        if (n <= 1) continue;
        const float inv = p.kv_scale / den;
        const int64_t row = p.q_rows != nullptr ? p.q_rows[b] : b;
        uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + (row * p.num_heads + kvh * p.group + ht * 16 + h) * D);
#pragma unroll
        for (int c = 0; c < PER / 2; ++c) dst[lane + 32 * c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
    }
}

template <int D, int NT>
cudaError_t launch_d(const Params &p, int blocks, bool combine, cudaStream_t stream) {
    constexpr int kWarps = warps_of(NT);
    constexpr int smem = kWarps * kStages * 2 * kUnit * fp4::row_bytes(D);
    static std::atomic<uint64_t> smem_set;
    auto kern = decode_fp4_split_kernel<D, NT>;
    cudaError_t e = smem_limit_once(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess || !combine) return e;
    cfg.gridDim = dim3(2 * kPlanSms);
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, decode_fp4_combine_kernel<D>, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

bool plan_decode_fp4(int batch, int num_heads, int num_kv_heads, int head_dim, int max_seq_len,
                     int sliding_window, DecodeFp4Plan *plan) {
    if (batch < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
        head_dim <= 0 || max_seq_len < 0)
        return false;
    DecodeFp4Plan p{};
    p.group = num_heads / num_kv_heads;
    p.head_tiles = (p.group + 15) / 16;
    p.tile_heads = p.group < 16 ? p.group : 16;
    int64_t span = max_seq_len;
    if (sliding_window > 0 && static_cast<int64_t>(sliding_window) + 15 < span)
        span = static_cast<int64_t>(sliding_window) + 15;
    const int64_t units = (span + kUnit - 1) / kUnit;
    const int64_t segments = static_cast<int64_t>(batch) * num_kv_heads * p.head_tiles;
    // Whole segments when they are short: one launch and no merge.
    p.whole = units <= kWholeUnits;
    const int64_t want = p.whole ? segments : (segments * units + kMinUnits - 1) / kMinUnits;
    const int warps = warps_of(p.group > 8 ? 2 : 1);
    // One block an SM, on as many SMs as there is work for; beyond that only whole segments.
    int64_t blocks = want < kPlanSms ? want : kPlanSms;
    if (p.whole && want > static_cast<int64_t>(kPlanSms) * warps) blocks = (want + warps - 1) / warps;
    if (blocks < 1) blocks = 1;
    if (blocks > 0x7fffffffLL / warps) return false;
    // Segments, rows and a warp's units are counted in 32 bits.
    if (segments > 0x7fffffffLL / 16 || segments * units / blocks > 0x3fffffff) return false;
    p.blocks = static_cast<int>(blocks);
    p.workers = p.blocks * warps;
    if (!p.whole)
        p.workspace_bytes = static_cast<size_t>(p.workers) * 2 * p.tile_heads * (head_dim + 2) * sizeof(float);
    *plan = p;
    return true;
}

cudaError_t launch_decode_fp4(const DecodeArgs &a, const DecodeFp4Plan &plan, cudaStream_t stream) {
    if (a.batch == 0) return cudaSuccess;
    Params p{};
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k_cache = static_cast<const uint8_t *>(a.k_cache);
    p.v_cache = static_cast<const uint8_t *>(a.v_cache);
    p.block_table = a.block_table;
    p.max_num_blocks = a.max_num_blocks;
    p.seq_lens = a.seq_lens;
    p.batch = a.batch;
    int log2_bs = 0;
    while ((1 << log2_bs) < a.block_size) ++log2_bs;
    p.log2_bs = log2_bs;
    const int64_t table_cap = static_cast<int64_t>(a.max_num_blocks) << log2_bs;
    p.seq_cap = table_cap < a.max_seq_len ? table_cap : a.max_seq_len;
    p.num_blocks = a.num_blocks;
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.group = plan.group;
    p.head_tiles = plan.head_tiles;
    p.window = a.sliding_window;
    p.scale_log2 = a.scale * a.kv_scale * kLog2e;
    p.kv_scale = a.kv_scale;
    p.workers = plan.workers;
    p.whole_units = plan.whole ? kWholeUnits : 0;
    p.tile_heads = plan.tile_heads;
    if (!plan.whole) p.pieces = static_cast<float *>(a.workspace);
    p.key = static_cast<const __nv_bfloat16 *>(a.key);
    p.value = static_cast<const __nv_bfloat16 *>(a.value);
    p.slot_mapping = a.slot_mapping;
    p.k_cache_w = static_cast<uint8_t *>(a.k_cache_w);
    p.v_cache_w = static_cast<uint8_t *>(a.v_cache_w);
    p.q_rows = a.q_rows;
    p.total_q = a.total_q;
    p.check_rows = a.check_rows ? 1 : 0;
    p.max_seqlen_q = a.max_seqlen_q;
    p.cu_k = a.cu_seqlens_k;
    p.after_prefill = a.after_prefill ? 1 : 0;
    p.err = a.err;
    const bool one = plan.group <= 8;
    switch (a.head_dim) {
        case 64: return one ? launch_d<64, 1>(p, plan.blocks, !plan.whole, stream)
                            : launch_d<64, 2>(p, plan.blocks, !plan.whole, stream);
        case 128: return one ? launch_d<128, 1>(p, plan.blocks, !plan.whole, stream)
                             : launch_d<128, 2>(p, plan.blocks, !plan.whole, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
