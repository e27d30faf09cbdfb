// decode_fp4.cu - decode over the 4-bit paged KV cache (fp4.cuh).
//
// For sequence b with L keys and query head h: out[b][h] = softmax(scale * q K^T) V over keys
// [max(0, L - w), L), K and V elements code * scale * kv_scale, read through block_table.
//
// A byte of cache holds 1.8 elements, so the kernel has to spend few instructions on each
// byte and keep the stream going without a pause:
//  * The keys of all (sequence, kv head, 16-head tile) segments are one flat list of 16-key
//    units, cut into equal ranges, one for each resident warp.  A warp streams its range
//    through its own ring of shared-memory stages without stopping at segment ends, so there
//    are no waves of blocks, no ragged tail and one pipeline fill a warp.
//  * One 16-key unit is 9 D contiguous bytes of K and of V (rows of codes and scales), each
//    moved by one bulk copy that a single lane issues.
//  * The products are f16 warp MMAs (m16n8k16, fp32 accumulate) with the unit's keys as the
//    M rows of S^T = K Q^T and the head dims as those of O^T += V^T P^T, the query heads the
//    8 columns of an n-tile (two n-tiles above 8 heads a kv head).  Codes become f16 by one
//    conversion for two and are scaled by one f16x2 product, exactly (fp4.cuh).
//  * The MMA's key and dim indices are permuted so that a lane needs whole groups of 16 dims:
//    K lane t of a quad takes groups t and t + 4 of its key rows; V lane group g owns dims
//    16 g .. 16 g + 15 (one scale a key) and keys 4 t .. 4 t + 3.  Loads are 8 bytes wide and,
//    with 72-byte rows, free of bank conflicts for V; and a lane ends up with 16 consecutive
//    dims of O for its heads, which it writes as whole vectors.
//  * A segment inside one warp's range is finished there.  A cut one leaves (m, l, O) of each
//    piece in the workspace and decode_fp4_combine_kernel (a programmatic dependent) merges
//    them.  When no sequence can be longer than kWholeUnits units, ranges are whole segments
//    and no combine is launched.
#include <math.h>

#include <atomic>

#include "decode_common.cuh"
#include "fp4.cuh"
#include "pa_common.cuh"
#include "pa_internal.h"
#include "sm100_ptx.cuh"

namespace pa {

namespace {

using namespace sm100;

constexpr int kWarps = 4;          // independent warps of a block
constexpr int kCtasPerSm = 4;      // resident blocks: 16 warps an SM
constexpr int kStages = 6;         // ring stages of a warp, one 16-key unit of K and V each
constexpr int kMinUnits = 8;       // smallest range of a warp (128 keys)
constexpr int kWholeUnits = 9;     // spans up to this many units are never cut
constexpr uint64_t kWaitNs = 2000000000ull;  // limit of a wait for a bulk copy

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
    int2 *cuts;        // [workers]: (segment, its last worker) if the first cut of it is here
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

// Units of sequence b and its key range; 0 units for a sequence that is not decoded here.
__device__ __forceinline__ int seq_units(const Params &p, int b, SeqRange &r, bool report) {
    if (p.q_rows != nullptr) {
        const int r0 = p.q_rows[b];
        const int sq = p.q_rows[b + 1] - r0;
        if (report && p.check_rows) {
            const int sk = p.seq_lens[b];
            if (sq < 0 || sq > p.max_seqlen_q || sq > sk) flag_error(p.err, kErrQueryLen);
            if (p.cu_k != nullptr && p.cu_k[b + 1] - p.cu_k[b] != sk) flag_error(p.err, kErrSeqlensK);
        }
        if (sq != 1 || r0 < 0 || r0 >= p.total_q) {
            if (report && sq == 1) flag_error(p.err, kErrQueryLen);
            r.L = r.start = r.base = 0;
            return -1;
        }
    }
    r = decode_range(p.seq_lens[b], p.seq_cap, p.window, 0, p.err, report);
    return (r.L - r.base + 15) >> 4;
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
    if constexpr (N == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
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

template <int D, int NT>
__device__ __forceinline__ void split_body(const Params &p) {
    constexpr int RB = fp4::row_bytes(D);
    constexpr int UB = 16 * RB;         // bytes of a unit of K (or V)
    constexpr int SB = 2 * UB;          // bytes of a stage
    constexpr int KC = D / 64;          // 16-dim groups of K a lane takes: t and t + 4
    constexpr int KSTEPS = D / 16;
    constexpr int VW = D / 64;          // words of V codes a lane takes of a key row
    constexpr int VD = 8 * VW;          // dims of V a lane owns
    constexpr int MT = D / 16;          // m-tiles of O^T

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kWarps * kStages];
    __shared__ long long part_sum[kWarps * 32];
    __shared__ long long s_total;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int HT = p.num_kv_heads * p.head_tiles;  // segments of a sequence
    const uint32_t ring = smem_u32(smem) + warp * kStages * SB;
    const uint32_t bar0 = smem_u32(&bars[warp * kStages]);
    const uint64_t policy = l2_policy_evict_first();

    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_barrier_init();
    }
    __syncwarp();

    // ---- this warp's range [f, f_end) of the flat unit list ----
    // Worker w of warp v of block c is v * blocks + c: few workers spread over many SMs.
    const int w = warp * gridDim.x + blockIdx.x;
    const int chunk = (p.batch + kWarps * 32 - 1) / (kWarps * 32);
    const bool report = blockIdx.x == 0;
    {
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
    long long range = 0;      // R: units a worker
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
        range = (total + p.workers - 1) / p.workers;
        if (range < kMinUnits) range = kMinUnits;
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
    long long todo = f < f_end ? f_end - f : 0;  // units this warp has to read
    if (p.cuts != nullptr && lane == 0) {
        // The first cut of a segment lies at the start of this range: its last worker.
        int2 cut = make_int2(-1, 0);
        if (todo > 0 && unit > 0 && unit <= range) {
            cut.x = seg.b * HT + seg.kvh * p.head_tiles + seg.ht;
            cut.y = static_cast<int>((f - unit + seg.units - 1) / range);
        }
        p.cuts[w] = cut;
    }

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

    // ---- the issue side: units ahead of the consumer, across segments ----
    Segment is = seg;
    int iu = unit;                 // next unit to issue
    long long ileft = todo;
    int blk_lane = -1;             // lane i: block of unit (iu_base + i) of segment is
    int iu_base = iu;
    auto load_blocks = [&]() {
        iu_base = iu;
        const int u = iu + lane;
        blk_lane = u < is.units
                       ? __ldg(p.block_table + static_cast<int64_t>(is.b) * p.max_num_blocks +
                               ((is.r.base + 16 * u) >> p.log2_bs))
                       : -1;
    };
    load_blocks();
    const int bs_mask = (1 << p.log2_bs) - 1;
    // Issue the next unit into stage st (all lanes call; lane 0 copies).
    auto issue = [&](int st) {
        if (iu == is.units) {  // next segment
            if (++is.ht == p.head_tiles) {
                is.ht = 0;
                if (++is.kvh == p.num_kv_heads) {
                    is.kvh = 0;
                    do {
                        ++is.b;
                        is.units = max(seq_units(p, is.b, is.r, false), 0);
                    } while (is.units == 0);
                }
            }
            iu = 0;
            load_blocks();
        } else if (iu - iu_base == 32) {
            load_blocks();
        }
        const int blk = __shfl_sync(0xffffffffu, blk_lane, iu - iu_base);
        const uint32_t bar = bar0 + 8 * st;
        const uint32_t dst = ring + st * SB;
        if (blk >= 0 && blk < p.num_blocks) {
            if (lane == 0) {
                const int64_t row = ((static_cast<int64_t>(blk) * p.num_kv_heads + is.kvh) << p.log2_bs) +
                                    ((is.r.base + 16 * iu) & bs_mask);
                mbar_arrive_expect_tx(bar, SB);
                bulk_load_policy(dst, p.k_cache + row * RB, UB, bar, policy);
                bulk_load_policy(dst + UB, p.v_cache + row * RB, UB, bar, policy);
            }
        } else {
            // A bad table entry reads as zeros.
            if (lane == 0) flag_error(p.err, kErrBlockRange);
            for (int i = lane; i < SB / 4; i += 32) sts_u32(dst + 4 * i, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        }
        ++iu;
        --ileft;
    };
#pragma unroll 1
    for (int s = 0; s < kStages && ileft > 0; ++s) issue(s);

    // ---- the consumer side ----
    // Q^T fragments of a segment: the B operand of S^T.  k-step ks is dims 4 (ks & 3) .. + 3 of
    // group t (ks < 4) or t + 4; head 8 j + g.  Heads past the group are zero.
    uint32_t qf[NT][KSTEPS][2];
    auto load_q = [&]() {
        const int rows_valid = min(16, p.group - seg.ht * 16);
        const int64_t row = p.q_rows != nullptr ? p.q_rows[seg.b] : seg.b;
        const __nv_bfloat16 *qb = p.q + (row * p.num_heads + seg.kvh * p.group + seg.ht * 16) * D;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
                if (8 * j + g < rows_valid) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        qb + (8 * j + g) * D + 16 * (t + 4 * c));
                    x[0] = __ldg(src);
                    x[1] = __ldg(src + 1);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    qf[j][4 * c + 2 * h][0] = bf16x2_to_f16x2(x[h].x);
                    qf[j][4 * c + 2 * h][1] = bf16x2_to_f16x2(x[h].y);
                    qf[j][4 * c + 2 * h + 1][0] = bf16x2_to_f16x2(x[h].z);
                    qf[j][4 * c + 2 * h + 1][1] = bf16x2_to_f16x2(x[h].w);
                }
            }
    };
    // O^T accumulators: tile i of 16 rows: row g is dim VD g + 2 i, row g + 8 dim VD g + 2 i + 1;
    // columns (heads) 8 j + 2 t and + 1.
    float o[NT][MT][4];
    // Per head: m_run is the reference maximum the weights are taken against (base 2); it moves
    // only when a score exceeds it by more than 8.  l_run sums this lane's keys.
    float m_run[NT][2], l_run[NT][2];
    auto reset = [&]() {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int i = 0; i < MT; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
            m_run[j][0] = m_run[j][1] = -INFINITY;
            l_run[j][0] = l_run[j][1] = 0.f;
        }
    };
    load_q();
    reset();
    int first_unit = unit;  // first unit of the segment's piece in this range

    // MMA row r of a unit is key 4 (r % 8 / 2) + r % 2 + 2 (r / 8): rows 2 t, 2 t + 1, 2 t + 8 and
    // 2 t + 9 are keys 4 t .. 4 t + 3.
    const int key_a = 4 * (g >> 1) + (g & 1);  // of row g; row g + 8 is key_a + 2
    const uint32_t k_off = key_a * RB, v_off = 4 * t * RB;

    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
#pragma unroll 1
    for (;;) {
        {
            uint64_t t0 = 0;
            for (uint32_t it = 0;; ++it) {
                const bool done = mbar_try_wait(bar0 + 8 * st, phase);
                if (__all_sync(0xffffffffu, done)) break;
                if ((it & 31u) == 31u) {
                    const uint64_t now = globaltimer_ns();
                    if (t0 == 0) t0 = now;
                    if (__any_sync(0xffffffffu, now - t0 > kWaitNs)) {
                        ok = false;
                        break;
                    }
                }
            }
            if (!ok) break;
        }
        const uint32_t kb = ring + st * SB;
        const uint32_t vb = kb + UB;
        const int key0 = seg.r.base + 16 * unit;
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
                const int blk = __ldg(p.block_table + static_cast<int64_t>(seg.b) * p.max_num_blocks +
                                      (pos >> p.log2_bs));
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
                        const uint32_t row = (which ? vb : kb) + (pos & 15) * RB;
                        sts_u32(row + 8 * gr, c.x);
                        sts_u32(row + 8 * gr + 4, c.y);
                        asm volatile("st.shared.u8 [%0], %1;" ::"r"(row + D / 2 + gr), "r"(sc) : "memory");
                    }
                }
                fence_proxy_async_smem();  // before the next copy into this stage
                __syncwarp();
            }
        }

        // S^T = K Q^T: even and odd k-steps in separate accumulators.
        float s[NT][4], s2[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = s2[j][e] = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            uint32_t wa[2], wb[2];  // 16 codes of rows g and g + 8
            if constexpr (D == 128) {
                lds_words<2>(kb + k_off + 8 * (t + 4 * c), wa);
                lds_words<2>(kb + k_off + 2 * RB + 8 * (t + 4 * c), wb);
            } else {  // 36-byte rows: 4-byte aligned
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t x[1];
                    lds_words<1>(kb + k_off + 8 * t + 4 * h, x);
                    wa[h] = x[0];
                    lds_words<1>(kb + k_off + 2 * RB + 8 * t + 4 * h, x);
                    wb[h] = x[0];
                }
            }
            const uint32_t sc = fp4::e4m3x2_to_f16x2(lds_u8(kb + k_off + D / 2 + t + 4 * c) |
                                                     (lds_u8(kb + k_off + 2 * RB + D / 2 + t + 4 * c) << 8));
            const uint32_t sa = __byte_perm(sc, 0u, 0x1010), sb = __byte_perm(sc, 0u, 0x3232);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t fa[4], fb[4];
                fp4::e2m1x8_to_f16x2x4(wa[h], fa);
                fp4::e2m1x8_to_f16x2x4(wb[h], fb);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t a[4] = {fp4::mul_f16x2(fa[2 * k], sa), fp4::mul_f16x2(fb[2 * k], sb),
                                           fp4::mul_f16x2(fa[2 * k + 1], sa),
                                           fp4::mul_f16x2(fb[2 * k + 1], sb)};
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        mma_f16_16816(k ? s2[j] : s[j], a, qf[j][4 * c + 2 * h + k][0],
                                      qf[j][4 * c + 2 * h + k][1]);
                }
            }
        }

        // V codes and scales of keys 4 t .. 4 t + 3.
        uint32_t vw[4][VW], vs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            lds_words<VW>(vb + v_off + k * RB + 4 * VW * g, vw[k]);
            vs[k] = lds_u8(vb + v_off + k * RB + D / 2 + (D == 128 ? g : g >> 1));
        }

        // Scale, mask (edge units only), online softmax per head column: elements 0, 1 are
        // key key_a, elements 2, 3 key key_a + 2; elements 0, 2 head 2t, 1, 3 head 2t+1.
        const bool edge = key0 < seg.r.start || key0 + 16 > seg.r.L;
        bool over = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = (s[j][e] + s2[j][e]) * p.scale_log2;
                if (edge) {
                    const int key = key0 + key_a + (e & 2);
                    if (key < seg.r.start || key >= seg.r.L) v = -INFINITY;
                }
                s[j][e] = v;
                over |= v > m_run[j][e & 1] + 8.f;
            }
        if (edge) {
            // Rows outside the range may hold anything: a zero scale makes them zeros.
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = key0 + 4 * t + k;
                if (key < seg.r.start || key >= seg.r.L) vs[k] = 0u;
            }
        }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float fr[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = fmaxf(s[j][e], s[j][e + 2]);
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    const float m_new = fmaxf(m_run[j][e], m);
                    const bool nd = m_new > m_run[j][e] + 8.f;
                    fr[e] = nd ? ex2_approx(m_run[j][e] - m_new) : 1.f;
                    l_run[j][e] *= fr[e];
                    if (nd) m_run[j][e] = m_new;
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[j][i][0] *= fr[0];
                    o[j][i][1] *= fr[1];
                    o[j][i][2] *= fr[0];
                    o[j][i][3] *= fr[1];
                }
            }
        }
        // P^T (B operand): f16 weights packed per key row and transposed; the denominator sums
        // the rounded weights that the MMA uses.
        uint32_t pb[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float m0 = m_run[j][0] == -INFINITY ? 0.f : m_run[j][0];
            const float m1 = m_run[j][1] == -INFINITY ? 0.f : m_run[j][1];
            const uint32_t w0 = pack_f16x2(ex2_approx(s[j][0] - m0), ex2_approx(s[j][1] - m1));
            const uint32_t w1 = pack_f16x2(ex2_approx(s[j][2] - m0), ex2_approx(s[j][3] - m1));
            add_f16x2_f32(l_run[j][0], l_run[j][1], w0);
            add_f16x2_f32(l_run[j][0], l_run[j][1], w1);
            pb[j][0] = movmatrix_trans(w0);  // keys 4 t, 4 t + 1
            pb[j][1] = movmatrix_trans(w1);  // keys 4 t + 2, 4 t + 3
        }
        // O^T += V^T P^T: the codes of two keys and one dim meet in a byte, low code first.
        const uint32_t s01 = fp4::e4m3x2_to_f16x2(vs[0] | (vs[1] << 8));
        const uint32_t s23 = fp4::e4m3x2_to_f16x2(vs[2] | (vs[3] << 8));
#pragma unroll
        for (int x = 0; x < VW; ++x) {
            constexpr uint32_t LO = 0x0f0f0f0fu;
            uint32_t f0[4], f1[4], f2[4], f3[4];
            fp4::e2m1x8_to_f16x2x4((vw[0][x] & LO) | ((vw[1][x] << 4) & ~LO), f0);  // even dims
            fp4::e2m1x8_to_f16x2x4(((vw[0][x] >> 4) & LO) | (vw[1][x] & ~LO), f1);  // odd dims
            fp4::e2m1x8_to_f16x2x4((vw[2][x] & LO) | ((vw[3][x] << 4) & ~LO), f2);
            fp4::e2m1x8_to_f16x2x4(((vw[2][x] >> 4) & LO) | (vw[3][x] & ~LO), f3);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a[4] = {fp4::mul_f16x2(f0[k], s01), fp4::mul_f16x2(f1[k], s01),
                                       fp4::mul_f16x2(f2[k], s23), fp4::mul_f16x2(f3[k], s23)};
#pragma unroll
                for (int j = 0; j < NT; ++j) mma_f16_16816(o[j][4 * x + k], a, pb[j][0], pb[j][1]);
            }
        }
        __syncwarp();
        if (ileft > 0) issue(st);
        if (++st == kStages) {
            st = 0;
            phase ^= 1u;
        }
        --todo;
        ++unit;
        if (!last_unit && todo > 0) continue;

        // ---- end of the segment's piece: lanes t hold heads 2 t, 2 t + 1 of each n-tile ----
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l_run[j][e] += __shfl_xor_sync(0xffffffffu, l_run[j][e], 4);
                l_run[j][e] += __shfl_xor_sync(0xffffffffu, l_run[j][e], 8);
                l_run[j][e] += __shfl_xor_sync(0xffffffffu, l_run[j][e], 16);
            }
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
                    const float inv = p.kv_scale / l_run[j][e];
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
                    if (g == 0) *reinterpret_cast<float2 *>(ph + D) = make_float2(m_run[j][e], l_run[j][e]);
                }
            }
        if (todo == 0) break;
        // Next segment.
        if (++seg.ht == p.head_tiles) {
            seg.ht = 0;
            if (++seg.kvh == p.num_kv_heads) {
                seg.kvh = 0;
                do {
                    ++seg.b;
                    seg.units = max(seq_units(p, seg.b, seg.r, false), 0);
                } while (seg.units == 0);
            }
        }
        unit = first_unit = 0;
        load_q();
        reset();
    }
    if (!ok) {
        // A copy never landed: flagged; give the copies in flight time to land, then leave.
        if (lane == 0) flag_error(p.err, kErrTimeout);
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? kCtasPerSm : 3)
    decode_fp4_split_kernel(const __grid_constant__ Params p) {
    griddep_launch_dependents();
    split_body<D, NT>(p);
    // As a programmatic dependent of the prefill kernel of the same call, this grid (and what
    // waits for it) completes after the prefill: its last block waits for the prefill grid.
    if (p.after_prefill && blockIdx.x == gridDim.x - 1) griddep_wait();
}

// Merge of the pieces of one cut segment, a block for each worker; the worker whose range
// starts at the segment's first cut does it.  With piece i holding (m_i, l_i, O_i):
//     M = max m_i,  out = kv_scale * sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
template <int D>
__global__ void __launch_bounds__(128) decode_fp4_combine_kernel(const __grid_constant__ Params p) {
    constexpr int PER = D / 32;
    griddep_wait();
    const int w = blockIdx.x;
    const int2 cut = p.cuts[w];
    if (cut.x < 0) return;
    const int HT = p.num_kv_heads * p.head_tiles;
    const int b = cut.x / HT;
    const int hs = cut.x - b * HT;
    const int kvh = hs / p.head_tiles, ht = hs - kvh * p.head_tiles;
    const int rows_valid = min(16, p.group - ht * 16);
    const int lane = threadIdx.x & 31;
    const int64_t row = p.q_rows != nullptr ? p.q_rows[b] : b;
    const int64_t stride = static_cast<int64_t>(p.tile_heads) * (D + 2);
    for (int h = threadIdx.x >> 5; h < rows_valid; h += 4) {
        // Piece 0 is the second one of worker w - 1; piece i the first one of worker w - 1 + i.
        auto piece = [&](int i) {
            return p.pieces + ((static_cast<int64_t>(w - 1 + i)) * 2 + (i == 0 ? 1 : 0)) * stride +
                   h * (D + 2);
        };
        const int n = cut.y - w + 2;
        float M = -INFINITY;
        for (int i = lane; i < n; i += 32) M = fmaxf(M, piece(i)[D]);
        M = warp_max(M);
        if (M == -INFINITY) M = 0.f;
        float acc[PER], den = 0.f;
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[k] = 0.f;
        for (int i0 = 0; i0 < n; i0 += 32) {
            float wt = 0.f;
            if (i0 + lane < n) {
                const float *ml = piece(i0 + lane) + D;
                wt = ex2_approx(ml[0] - M);
                den += wt * ml[1];
            }
            const int m = min(32, n - i0);
#pragma unroll 4
            for (int k = 0; k < m; ++k) {
                const float x = __shfl_sync(0xffffffffu, wt, k);
                const float2 *src = reinterpret_cast<const float2 *>(piece(i0 + k)) + lane * (PER / 2);
#pragma unroll
                for (int c = 0; c < PER / 2; ++c) {
                    const float2 v = src[c];
                    acc[2 * c] += x * v.x;
                    acc[2 * c + 1] += x * v.y;
                }
            }
        }
        den = warp_sum(den);
        const float inv = p.kv_scale / den;
        uint32_t *dst = reinterpret_cast<uint32_t *>(
            p.out + (row * p.num_heads + kvh * p.group + ht * 16 + h) * D + lane * PER);
#pragma unroll
        for (int c = 0; c < PER / 2; ++c) dst[c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
    }
}

template <int D, int NT>
cudaError_t launch_d(const Params &p, int blocks, bool combine, cudaStream_t stream) {
    constexpr int smem = kWarps * kStages * 2 * 16 * fp4::row_bytes(D);
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
    cfg.numAttrs = p.after_prefill ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess || !combine) return e;
    cfg.gridDim = dim3(p.workers);
    cfg.blockDim = dim3(128);
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
    const int64_t units = (span + 15) / 16;
    const int64_t segments = static_cast<int64_t>(batch) * num_kv_heads * p.head_tiles;
    // Whole segments when they are short: one launch and no merge.
    p.whole = units <= kWholeUnits;
    const int64_t want = p.whole ? segments : (segments * units + kMinUnits - 1) / kMinUnits;
    int64_t blocks = (want + kWarps - 1) / kWarps;
    const int64_t resident = static_cast<int64_t>(kPlanSms) * (p.group > 8 ? 3 : kCtasPerSm);
    if (!p.whole && blocks > resident) blocks = resident;
    if (blocks < 1) blocks = 1;
    if (blocks > 0x7fffffffLL / kWarps) return false;
    p.blocks = static_cast<int>(blocks);
    p.workers = p.blocks * kWarps;
    if (!p.whole) {
        p.pieces_bytes = (static_cast<size_t>(p.workers) * 2 * p.tile_heads * (head_dim + 2) * sizeof(float) + 255) / 256 * 256;
        p.workspace_bytes = p.pieces_bytes + static_cast<size_t>(p.workers) * sizeof(int2);
    }
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
    if (!plan.whole) {
        p.pieces = static_cast<float *>(a.workspace);
        p.cuts = reinterpret_cast<int2 *>(static_cast<uint8_t *>(a.workspace) + plan.pieces_bytes);
    }
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
