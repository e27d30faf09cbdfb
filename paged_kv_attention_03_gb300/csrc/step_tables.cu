// step_tables.cu - the metadata of a serving step built on the GPU from the requests' lengths:
// block tables, slots, positions, lengths and offsets, with the pool's free blocks kept as a
// stack in device memory; and the release of finished requests' blocks.
//
// prepare: with c_i cached and q_i new tokens of request i and blocks of B tokens,
//     have_i = ceil(c_i / B),  need_i = ceil((c_i + q_i) / B) - have_i,
//     cu = exclusive prefix sum of q,  off = exclusive prefix sum of need,
//     block_table[i][have_i + k] = free[n_free - 1 - off_i - k],  0 <= k < need_i,
//     token t of request i: position p = c_i + t - cu_i, slot block_table[i][p / B] * B + p % B.
// release: the entries [0, ceil(len_i / B)) of finished rows follow free[n_free) in row order;
//     entries that are no block ids are left out (a flagged call).
//
// The data is a few bytes a token, so the time is launches and dependent loads.  Every block
// scans all requests by itself (at most kMaxStepSeqs, two words of shared memory each) and
// takes its share of the tokens, so no block waits for another.  A thread takes four
// consecutive tokens: one binary search in shared memory and 16-byte stores; a token's block
// comes straight from the free list, and the first token of each new block writes the table
// entry.  What a caller may update in place (lengths, the free count) is written when no
// block reads it any more: by the same block when there is one, else by a second launch, a
// programmatic dependent that repeats the scan while the first runs.
//
// Measured (replayed from a graph): 64 decodes 4.6 us in one launch; 2033 requests with 526k
// slots 8.6 us in two; the release of a seventh of 64 requests 4.0 us, of half of 1024 5.9 (a call
// from Python takes the host 9-12 us).
#include <algorithm>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "sm100_ptx.cuh"

namespace pa {

namespace {

constexpr int kThreads = 512;
// Items (tokens or table entries) up to which one block does all of a call, four a thread.  One
// launch / two: 64 requests of a token 4.7 / 5.3 us, 1024 of one 5.8 / 6.8, 64 of 48 6.7 / 5.6.
constexpr int64_t kAloneItems = 4 * kThreads;

// Sums saturate at 2^31 - 1: they are offsets into arrays of fewer items, and a saturated sum
// of non-negative numbers does not depend on the order.
constexpr uint32_t kTop = 0x7fffffffu;
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return min(a + b, kTop); }

// One request: tokens (prepare) or entries (release), and new blocks.
struct Need {
    uint32_t items;
    uint32_t blocks;
};

__device__ __forceinline__ uint32_t table_cap(const StepArgs &a) {
    const uint64_t cap = static_cast<uint64_t>(a.max_num_blocks) << a.log2_bs;
    return static_cast<uint32_t>(min(cap, static_cast<uint64_t>(kTop)));
}

// Cached tokens of request i, inside [0, capacity of its row].
__device__ __forceinline__ uint32_t cached(const StepArgs &a, int i) {
    return min(static_cast<uint32_t>(max(a.context_lens[i], 0)), table_cap(a));
}

// New blocks of a request with c cached and q new tokens.
__device__ __forceinline__ uint32_t new_blocks(const StepArgs &a, uint32_t c, uint32_t q) {
    const uint32_t up = (1u << a.log2_bs) - 1u;
    const uint32_t len = min(c + q, table_cap(a));  // below 2^32
    return ((len + up) >> a.log2_bs) - ((c + up) >> a.log2_bs);
}

template <bool PREPARE>
__device__ __forceinline__ Need need_of(const StepArgs &a, int i, bool report) {
    Need n;
    const uint32_t cap = table_cap(a);
    if constexpr (PREPARE) {
        const int c_raw = a.context_lens[i], q_raw = a.query_lens[i];
        const uint32_t c = cached(a, i);
        n.items = static_cast<uint32_t>(max(q_raw, 0));
        n.blocks = new_blocks(a, c, n.items);
        if (report) {
            if (c_raw < 0 || static_cast<uint32_t>(c_raw) > cap || c + n.items > cap)
                flag_error(a.err, kErrSeqRange);
            if (q_raw < 0) flag_error(a.err, kErrQueryLen);
        }
    } else {
        const int raw = a.seq_lens[i];
        const bool done = a.finished[i] != 0;
        const uint32_t len = min(static_cast<uint32_t>(max(raw, 0)), cap);
        n.items = done ? (len + (1u << a.log2_bs) - 1u) >> a.log2_bs : 0u;
        n.blocks = 0;
        if (report && done && (raw < 0 || static_cast<uint32_t>(raw) > cap)) flag_error(a.err, kErrSeqRange);
    }
    return n;
}

// Exclusive prefix sums of all requests' needs into shared memory (n + 1 words each): the needs
// by coalesced loads, then a thread sums a run of them (of odd length: no bank conflicts).
// (Runs read from global memory took 76 us for 16384 requests.)
template <bool PREPARE>
__device__ __forceinline__ void scan(const StepArgs &a, uint32_t *items, uint32_t *blocks, bool report) {
    __shared__ uint32_t wsum[2][kThreads / 32];
    const int n = a.num_seqs;
    const int per = ((n + kThreads - 1) / kThreads) | 1;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const Need x = need_of<PREPARE>(a, i, report);
        items[i] = x.items;
        if (PREPARE) blocks[i] = x.blocks;
    }
    __syncthreads();
    const int i0 = min(n, static_cast<int>(threadIdx.x) * per), i1 = min(n, i0 + per);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t si = 0, sb = 0;
    for (int i = i0; i < i1; ++i) {
        si = add_sat(si, items[i]);
        if (PREPARE) sb = add_sat(sb, blocks[i]);
    }
    uint32_t pi = si, pb = sb;  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, pi, o), y = __shfl_up_sync(0xffffffffu, pb, o);
        if (lane >= o) {
            pi = add_sat(pi, x);
            pb = add_sat(pb, y);
        }
    }
    if (lane == 31) {
        wsum[0][warp] = pi;
        wsum[1][warp] = pb;
    }
    uint32_t ei = __shfl_up_sync(0xffffffffu, pi, 1), eb = __shfl_up_sync(0xffffffffu, pb, 1);
    if (lane == 0) ei = eb = 0;
    __syncthreads();
    for (int k = 0; k < warp; ++k) {
        ei = add_sat(ei, wsum[0][k]);
        eb = add_sat(eb, wsum[1][k]);
    }
    for (int i = i0; i < i1; ++i) {
        const uint32_t x = items[i];
        items[i] = ei;
        ei = add_sat(ei, x);
        if (PREPARE) {
            const uint32_t y = blocks[i];
            blocks[i] = eb;
            eb = add_sat(eb, y);
        }
    }
    if (threadIdx.x == kThreads - 1) {  // (its run is the last one, or empty)
        items[n] = ei;
        if (PREPARE) blocks[n] = eb;
    }
    __syncthreads();
    // More tokens than max_tokens: what is beyond is no token of any request, so that no block is
    // taken for it (a flagged call, its second sum is left to one thread).
    const uint32_t most = static_cast<uint32_t>(a.max_tokens);
    if (PREPARE && items[n] > most) {
        for (int i = threadIdx.x; i < n; i += kThreads)
            blocks[i] = new_blocks(a, cached(a, i), min(items[i + 1], most) - min(items[i], most));
        __syncthreads();
        for (int i = threadIdx.x; i <= n; i += kThreads) items[i] = min(items[i], most);
        if (threadIdx.x == 0) {
            uint32_t sum = 0;
            for (int i = 0; i < n; ++i) {
                const uint32_t x = blocks[i];
                blocks[i] = sum;
                sum = add_sat(sum, x);
            }
            blocks[n] = sum;
            if (report) flag_error(a.err, kErrQueryLen);
        }
        __syncthreads();
    }
}

// The last request whose first item is at or before k (k below the total): the one that holds k.
__device__ __forceinline__ int holder(const uint32_t *items, int n, uint32_t k) {
    int lo = 0, hi = n;  // items[lo] <= k < items[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (items[m] <= k)
            lo = m;
        else
            hi = m;
    }
    return lo;
}

// The free count, inside [0, num_blocks].
__device__ __forceinline__ uint32_t free_count(const StepArgs &a, bool report) {
    const int raw = *a.num_free;
    if (report && (raw < 0 || raw > a.num_blocks)) flag_error(a.err, kErrBlockRange);
    return static_cast<uint32_t>(min(static_cast<int64_t>(max(raw, 0)), a.num_blocks));
}

__device__ __forceinline__ void store4(int32_t *dst, int64_t k, int64_t end, const int (&v)[4]) {
    if (k + 4 <= end && (reinterpret_cast<uintptr_t>(dst + k) & 15u) == 0) {
        *reinterpret_cast<int4 *>(dst + k) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k + j < end) dst[k + j] = v[j];
    }
}

// Slots, positions and new table entries of this block's tokens.
__device__ __forceinline__ void tokens(const StepArgs &a, const uint32_t *cu, const uint32_t *off) {
    const int n = a.num_seqs;
    const uint32_t total = n > 0 ? cu[n] : 0u;
    const uint32_t nfree = free_count(a, false);
    const uint32_t cap = table_cap(a);
    const uint32_t up = (1u << a.log2_bs) - 1u;
    const int64_t stride = 4ll * kThreads * gridDim.x;
    for (int64_t t0 = 4ll * (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x);
         t0 < a.max_tokens; t0 += stride) {
        int slot[4], posv[4];
        int seq = -1;
        uint32_t begin = 0, end = 0, c = 0, have = 0, cur_blk = 0xffffffffu;
        int entry = -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            slot[j] = -1;  // past the last token: padding
            posv[j] = 0;
            const int64_t tt = t0 + j;
            if (tt >= total) continue;
            const uint32_t t = static_cast<uint32_t>(tt);
            if (seq < 0 || t >= end) {
                // Often the next request; else (empty ones between) search again.
                if (seq >= 0 && t < cu[seq + 2 <= n ? seq + 2 : n])
                    ++seq;
                else
                    seq = holder(cu, n, t);
                begin = cu[seq];
                end = cu[seq + 1];
                c = cached(a, seq);
                have = (c + up) >> a.log2_bs;
                cur_blk = 0xffffffffu;
            }
            const uint32_t pos = c + (t - begin);  // below 2^32
            posv[j] = static_cast<int>(min(pos, kTop));
            if (pos >= cap) continue;  // no room in the row (flagged by the scan)
            const uint32_t blk = pos >> a.log2_bs;
            int32_t *at = a.block_table + static_cast<int64_t>(seq) * a.max_num_blocks + blk;
            if (blk != cur_blk) {
                cur_blk = blk;
                const bool fresh = blk >= have;
                if (fresh) {
                    const uint32_t rank = add_sat(off[seq], blk - have);
                    entry = rank < nfree ? a.free_blocks[nfree - 1 - rank] : -1;
                } else {
                    entry = *at;
                }
                if (entry < 0 || entry >= a.num_blocks) {
                    // Out of blocks is flagged where the count is; other entries are bad ones.
                    if (!fresh || add_sat(off[seq], blk - have) < nfree) flag_error(a.err, kErrBlockRange);
                    entry = -1;
                }
            }
            if ((pos & up) == 0) *at = entry;  // the first token of a block: the block is new
            if (entry >= 0) slot[j] = (entry << a.log2_bs) | static_cast<int>(pos & up);
        }
        store4(a.slot_mapping, t0, a.max_tokens, slot);
        if (a.positions != nullptr) store4(a.positions, t0, a.max_tokens, posv);
    }
}

// Lengths, offsets and the free count.
__device__ __forceinline__ void publish_prepare(const StepArgs &a, const uint32_t *cu,
                                                const uint32_t *off) {
    const int n = a.num_seqs;
    const uint32_t nfree = free_count(a, true);
    const uint32_t up = (1u << a.log2_bs) - 1u;
    const uint32_t cap = table_cap(a);
    const uint32_t used = min(n > 0 ? off[n] : 0u, nfree);
    if (threadIdx.x == 0) {
        if (n > 0 && off[n] > nfree) flag_error(a.err, kErrNoBlocks);
        a.cu_seqlens_q[n] = n > 0 ? static_cast<int>(cu[n]) : 0;
    }
    __syncthreads();  // the count has been read by all (num_free_out may be num_free)
    if (threadIdx.x == 0) *a.num_free_out = static_cast<int>(nfree - used);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t c = cached(a, i);
        uint32_t len = min(c + (cu[i + 1] - cu[i]), cap);
        // Out of blocks: the sequence ends where its last block does.
        const uint32_t have = (c + up) >> a.log2_bs;
        const uint32_t got = off[i] < nfree ? nfree - off[i] : 0u;
        const uint64_t room = static_cast<uint64_t>(have + static_cast<uint64_t>(got)) << a.log2_bs;
        if (room < len) len = static_cast<uint32_t>(room);
        a.seq_lens_out[i] = static_cast<int>(len);
        a.cu_seqlens_q[i] = static_cast<int>(cu[i]);
    }
}

// A release in two launches that meets an entry that is no block id sets its mark, which tells the
// second launch to append the entries anew, without such ones.  Calls take the marks in turn, and a
// mark stays set: clearing it could come between the launches of another stream's call.  So after
// a bad call one in kMarks takes the slow way too (262k entries: 262 us against 7), as do replays
// of a captured one.
constexpr int kMarks = 4096;
__device__ unsigned bad_entries[kMarks];

// The table entries of four consecutive released items k0 .. k0 + 3; -1 past the total.
__device__ __forceinline__ void released(const StepArgs &a, const uint32_t *first, uint32_t total,
                                         uint32_t k0, int (&entry)[4]) {
    int seq = -1;
    uint32_t begin = 0, end = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        entry[j] = -1;
        const uint32_t k = k0 + j;
        if (k >= total) continue;
        if (seq < 0 || k >= end) {
            seq = holder(first, a.num_seqs, k);
            begin = first[seq];
            end = first[seq + 1];
        }
        entry[j] = a.block_table[static_cast<int64_t>(seq) * a.max_num_blocks + (k - begin)];
    }
}

__device__ __forceinline__ bool is_block(const StepArgs &a, int entry) {
    return entry >= 0 && entry < a.num_blocks;
}

// This block's released entries to the end of the free list, each at its place among all of them:
// whether that holds for this thread's, or one of them is no block id.
__device__ __forceinline__ bool push_blocks(const StepArgs &a, const uint32_t *first) {
    const int n = a.num_seqs;
    const uint32_t total = n > 0 ? first[n] : 0u;
    const uint32_t nfree = free_count(a, false);
    const int64_t stride = 4ll * kThreads * gridDim.x;
    bool good = true;
    for (int64_t k0 = 4ll * (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x); k0 < total;
         k0 += stride) {
        int entry[4];
        released(a, first, total, static_cast<uint32_t>(k0), entry);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (k0 + j >= total) continue;
            const int64_t dst = static_cast<int64_t>(nfree) + k0 + j;
            const bool id = is_block(a, entry[j]);
            if (!id || dst >= a.num_blocks) flag_error(a.err, kErrBlockRange);
            good = good && id;
            if (id && dst < a.num_blocks) a.free_blocks[dst] = entry[j];
        }
    }
    return good;
}

// One block appends all released entries that are block ids, one behind the other; how many.
__device__ __forceinline__ uint32_t push_blocks_only(const StepArgs &a, const uint32_t *first,
                                                     uint32_t nfree) {
    __shared__ uint32_t wcount[kThreads / 32];
    const uint32_t total = a.num_seqs > 0 ? first[a.num_seqs] : 0u;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t kept = 0;
    for (uint32_t k0 = 0; k0 < total; k0 += 4 * kThreads) {  // (below 2^32: total is below 2^31)
        int entry[4];
        released(a, first, total, k0 + 4 * threadIdx.x, entry);
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) mine += is_block(a, entry[j]) ? 1u : 0u;
        uint32_t inc = mine;  // inclusive over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        __syncthreads();  // the previous round's counts have been read
        if (lane == 31) wcount[warp] = inc;
        __syncthreads();
        int64_t dst = static_cast<int64_t>(nfree) + kept + (inc - mine);
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) dst += wcount[w];
            kept += wcount[w];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!is_block(a, entry[j])) continue;
            if (dst < a.num_blocks) a.free_blocks[dst] = entry[j];
            ++dst;
        }
    }
    return kept;
}

// again: not every entry was at its place.
__device__ __forceinline__ void publish_release(const StepArgs &a, const uint32_t *first, bool again) {
    const int n = a.num_seqs;
    const uint32_t nfree = free_count(a, true);
    uint32_t total = n > 0 ? first[n] : 0u;
    if (again) total = push_blocks_only(a, first, nfree);
    __syncthreads();
    if (threadIdx.x == 0)
        *a.num_free_out = static_cast<int>(min(static_cast<int64_t>(nfree) + total, a.num_blocks));
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int len = a.seq_lens[i];
        a.seq_lens_out[i] = a.finished[i] != 0 ? 0 : len;
    }
}

enum : int { kAll = 0, kItems = 1, kPublish = 2 };

// PART kItems: the first launch of two; kPublish: the second; kAll: one block does both.
template <bool PREPARE, int PART>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepArgs a) {
    extern __shared__ uint32_t sums[];
    uint32_t *items = sums, *blocks = sums + a.num_seqs + 1;
    if constexpr (PART == kItems) sm100::griddep_launch_dependents();
    scan<PREPARE>(a, items, blocks, PART != kItems);
    bool again = false;
    if constexpr (PART != kPublish) {
        if constexpr (PREPARE)
            tokens(a, items, blocks);
        else
            again = !push_blocks(a, items);
    }
    if constexpr (!PREPARE && PART == kItems)
        if (again) atomicExch(&bad_entries[a.mark], 1u);
    if constexpr (PART == kAll) again = __syncthreads_or(again);
    if constexpr (PART == kPublish) {
        sm100::griddep_wait();
        if constexpr (!PREPARE) again = __ldcg(&bad_entries[a.mark]) != 0u;
    }
    if constexpr (PART != kItems) {
        if constexpr (PREPARE)
            publish_prepare(a, items, blocks);
        else
            publish_release(a, items, again);
    }
}

template <bool PREPARE, int PART>
cudaError_t launch_part(const StepArgs &a, int blocks, cudaStream_t stream) {
    const int smem = (a.num_seqs + 1) * (PREPARE ? 2 : 1) * 4;
    auto kern = step_kernel<PREPARE, PART>;
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> smem_set;
        const cudaError_t e = smem_limit_once(kern, (kMaxStepSeqs + 1) * (PREPARE ? 2 : 1) * 4, smem_set);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PART == kPublish ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool PREPARE>
cudaError_t launch_step(const StepArgs &a, int64_t items, cudaStream_t stream) {
    if (items <= kAloneItems) return launch_part<PREPARE, kAll>(a, 1, stream);
    const int64_t want = (items + 4 * kThreads - 1) / (4 * kThreads);
    const cudaError_t e =
        launch_part<PREPARE, kItems>(a, static_cast<int>(std::min<int64_t>(want, kPlanSms)), stream);
    return e != cudaSuccess ? e : launch_part<PREPARE, kPublish>(a, 1, stream);
}

}  // namespace

cudaError_t launch_prepare_step(const StepArgs &a, cudaStream_t stream) {
    return launch_step<true>(a, a.max_tokens, stream);
}

cudaError_t launch_release_blocks(const StepArgs &args, cudaStream_t stream) {
    static std::atomic<unsigned> calls{0};
    StepArgs a = args;
    a.mark = static_cast<int>(calls.fetch_add(1, std::memory_order_relaxed) % kMarks);
    // The released entries are at most the whole table and at most the pool.
    return launch_step<false>(a, std::min<int64_t>(static_cast<int64_t>(a.num_seqs) * a.max_num_blocks, a.num_blocks), stream);
}

}  // namespace pa
