// pa_api_step.cu - the extern "C" boundary of the serving step over a 4-bit cache: block
// tables and slots (step_tables.cu), the quantising store and its inverse (store_fp4.cu),
// decode (decode_fp4.cu) and packed prefill (prefill.cu).  Host-side argument validation only.
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "pa_gb300.h"
#include "pa_internal.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

// kv_scale of a 4-bit cache: the scales times it stay far enough inside the normal fp32 range
// that quotients by them and their remainders keep all bits.
bool fp4_scale_ok(float s) { return s >= 1e-25f && s <= 1e25f; }

// Longest sequence: positions past its end, up to a list of units, stay inside 32 bits.
constexpr int kMostKeys = 0x7ffff000;

// Sizes of a 4-bit cache: PA_OK, or why it is refused.
pa_status check_fp4_cache(int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                          float kv_scale) {
    if (num_blocks < 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0 || !fp4_scale_ok(kv_scale))
        return PA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (!is_pow2(block_size) || block_size < 16 || block_size > 256) return PA_ERR_UNSUPPORTED;
    if (num_blocks * block_size > 0x7fffff00LL) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// Sizes shared by decode and prefill.
pa_status check_fp4_heads(int num_heads, int num_kv_heads, float scale, float kv_scale) {
    if (num_heads <= 0 || num_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    // (scale * kv_scale * log2 e is one factor in the kernels.)
    if (!(scale > 0.f) || !(scale * kv_scale < 1.0e38f)) return PA_ERR_INVALID_ARG;
    if (num_heads / num_kv_heads > 64) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

pa_status run_store_fp4(const void *key, const void *value, void *k_cache, void *v_cache,
                        const int32_t *slot_mapping, int64_t num_tokens, int64_t num_blocks,
                        int block_size, int num_kv_heads, int head_dim, float kv_scale,
                        cudaStream_t stream) {
    pa::StoreArgs a{};
    a.key = key;
    a.value = value;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.slot_mapping = slot_mapping;
    a.num_tokens = num_tokens;
    a.num_slots = num_blocks * block_size;
    a.err = pa::device_error_word();
    return pa::cuda_status(pa::launch_store_kvcache_fp4(a, num_kv_heads, head_dim, log2_of(block_size), kv_scale, stream));
}

// The step's shared arguments.
pa_status check_step(const int32_t *block_table, int max_num_blocks, int num_seqs,
                     const int32_t *free_blocks, const int32_t *num_free,
                     const int32_t *num_free_out, int64_t num_blocks, int block_size) {
    if (num_seqs < 0 || max_num_blocks < 0 || num_blocks < 0 || block_size <= 0) return PA_ERR_INVALID_ARG;
    if (!is_pow2(block_size) || block_size > 1024) return PA_ERR_UNSUPPORTED;
    if (num_seqs > pa::kMaxStepSeqs) return PA_ERR_UNSUPPORTED;
    if (num_blocks * block_size > 0x7fffff00LL) return PA_ERR_UNSUPPORTED;  // slots are int32
    if (!num_free || !num_free_out || (num_blocks > 0 && !free_blocks)) return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!block_table || max_num_blocks == 0)) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_prepare_step(int32_t *block_table, int32_t *seq_lens, int32_t *cu_seqlens_q,
                          int32_t *slot_mapping, int32_t *positions, int32_t *num_free_out,
                          const int32_t *context_lens, const int32_t *query_lens,
                          const int32_t *free_blocks, const int32_t *num_free, int num_seqs,
                          int max_num_blocks, int64_t max_tokens, int64_t num_blocks,
                          int block_size, void *stream) {
    const pa_status st = check_step(block_table, max_num_blocks, num_seqs, free_blocks, num_free,
                                    num_free_out, num_blocks, block_size);
    if (st != PA_OK) return st;
    if (max_tokens < 0 || max_tokens > 0x7fffff00LL || !cu_seqlens_q || (max_tokens > 0 && !slot_mapping))
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!seq_lens || !context_lens || !query_lens)) return PA_ERR_INVALID_ARG;
    pa::StepArgs a{};
    a.block_table = block_table;
    a.max_num_blocks = max_num_blocks;
    a.num_seqs = num_seqs;
    a.log2_bs = log2_of(block_size);
    a.free_blocks = const_cast<int32_t *>(free_blocks);
    a.num_free = num_free;
    a.num_free_out = num_free_out;
    a.num_blocks = num_blocks;
    a.context_lens = context_lens;
    a.query_lens = query_lens;
    a.cu_seqlens_q = cu_seqlens_q;
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.max_tokens = max_tokens;
    a.seq_lens_out = seq_lens;
    a.err = pa::device_error_word();
    return pa::cuda_status(pa::launch_prepare_step(a, static_cast<cudaStream_t>(stream)));
}

pa_status pa_release_blocks(int32_t *free_blocks, int32_t *num_free_out, int32_t *seq_lens_out,
                            const int32_t *finished, const int32_t *seq_lens,
                            const int32_t *block_table, const int32_t *num_free, int num_seqs,
                            int max_num_blocks, int64_t num_blocks, int block_size, void *stream) {
    const pa_status st = check_step(block_table, max_num_blocks, num_seqs, free_blocks, num_free,
                                    num_free_out, num_blocks, block_size);
    if (st != PA_OK) return st;
    if (num_seqs > 0 && (!finished || !seq_lens || !seq_lens_out)) return PA_ERR_INVALID_ARG;
    pa::StepArgs a{};
    a.block_table = const_cast<int32_t *>(block_table);
    a.max_num_blocks = max_num_blocks;
    a.num_seqs = num_seqs;
    a.log2_bs = log2_of(block_size);
    a.free_blocks = free_blocks;
    a.num_free = num_free;
    a.num_free_out = num_free_out;
    a.num_blocks = num_blocks;
    a.finished = finished;
    a.seq_lens = seq_lens;
    a.seq_lens_out = seq_lens_out;
    a.err = pa::device_error_word();
    return pa::cuda_status(pa::launch_release_blocks(a, static_cast<cudaStream_t>(stream)));
}

pa_status pa_store_kvcache_fp4(const void *key, const void *value, void *k_cache, void *v_cache,
                               const int32_t *slot_mapping, int64_t num_tokens,
                               int64_t num_blocks, int block_size, int num_kv_heads,
                               int head_dim, float kv_scale, void *stream) {
    if (num_tokens < 0) return PA_ERR_INVALID_ARG;
    const pa_status st = check_fp4_cache(num_blocks, block_size, num_kv_heads, head_dim, kv_scale);
    if (st != PA_OK || num_tokens == 0) return st;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return PA_ERR_INVALID_ARG;
    return run_store_fp4(key, value, k_cache, v_cache, slot_mapping, num_tokens, num_blocks, block_size,
                         num_kv_heads, head_dim, kv_scale, static_cast<cudaStream_t>(stream));
}

pa_status pa_gather_kvcache_fp4(void *key, void *value, const void *k_cache, const void *v_cache,
                                const int32_t *slot_mapping, int64_t num_tokens,
                                int64_t num_blocks, int block_size, int num_kv_heads,
                                int head_dim, float kv_scale, void *stream) {
    if (num_tokens < 0) return PA_ERR_INVALID_ARG;
    const pa_status st = check_fp4_cache(num_blocks, block_size, num_kv_heads, head_dim, kv_scale);
    if (st != PA_OK || num_tokens == 0) return st;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return PA_ERR_INVALID_ARG;
    pa::GatherArgs a{};
    a.key = key;
    a.value = value;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.slot_mapping = slot_mapping;
    a.num_tokens = num_tokens;
    a.num_slots = num_blocks * block_size;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.log2_bs = log2_of(block_size);
    a.kv_scale = kv_scale;
    a.err = pa::device_error_word();
    return pa::cuda_status(pa::launch_gather_kvcache_fp4(a, static_cast<cudaStream_t>(stream)));
}

size_t pa_decode_fp4_workspace_size(int batch, int num_heads, int num_kv_heads, int head_dim,
                                    int max_seq_len, int sliding_window) {
    pa::DecodeFp4Plan plan;
    if (!pa::plan_decode_fp4(batch, num_heads, num_kv_heads, head_dim, max_seq_len, sliding_window, &plan))
        return 0;
    return plan.workspace_bytes;
}

pa_status pa_decode_fp4(void *out, const void *q, const void *key, const void *value,
                        const int32_t *slot_mapping, void *k_cache, void *v_cache,
                        const int32_t *block_table, int max_num_blocks, const int32_t *seq_lens,
                        int batch, int max_seq_len, int64_t num_blocks, int block_size,
                        int num_heads, int num_kv_heads, int head_dim, int sliding_window,
                        float scale, float kv_scale, void *workspace, size_t workspace_bytes,
                        void *stream) {
    if (batch < 0 || max_seq_len < 0 || max_num_blocks < 0) return PA_ERR_INVALID_ARG;
    if (max_seq_len > kMostKeys) return PA_ERR_UNSUPPORTED;
    pa_status st = check_fp4_cache(num_blocks, block_size, num_kv_heads, head_dim, kv_scale);
    if (st == PA_OK) st = check_fp4_heads(num_heads, num_kv_heads, scale, kv_scale);
    if (st != PA_OK) return st;
    if (batch > 65535) return PA_ERR_UNSUPPORTED;
    const bool has_new = key || value || slot_mapping;
    if (has_new && !(key && value && slot_mapping)) return PA_ERR_INVALID_ARG;
    if (batch == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_table || !seq_lens) return PA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        (has_new && (!aligned(key, 16) || !aligned(value, 16))))
        return PA_ERR_INVALID_ARG;
    if (max_seq_len > 0 && max_num_blocks == 0) return PA_ERR_INVALID_ARG;
    pa::DecodeFp4Plan plan;
    if (!pa::plan_decode_fp4(batch, num_heads, num_kv_heads, head_dim, max_seq_len, sliding_window, &plan))
        return PA_ERR_INVALID_ARG;
    if (plan.workspace_bytes > 0 &&
        (!workspace || workspace_bytes < plan.workspace_bytes || !aligned(workspace, 256)))
        return PA_ERR_INVALID_ARG;
    pa::DecodeArgs a{};
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.max_num_blocks = max_num_blocks;
    a.seq_lens = seq_lens;
    a.batch = batch;
    a.max_seq_len = max_seq_len;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.sliding_window = sliding_window;
    a.scale = scale;
    a.kv_scale = kv_scale;
    a.workspace = workspace;
    a.key = key;
    a.value = value;
    a.slot_mapping = slot_mapping;
    a.k_cache_w = k_cache;
    a.v_cache_w = v_cache;
    a.err = pa::device_error_word();
    return pa::cuda_status(pa::launch_decode_fp4(a, plan, static_cast<cudaStream_t>(stream)));
}

size_t pa_varlen_prefill_fp4_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                            int head_dim, int max_seqlen_k, int sliding_window) {
    pa::DecodeFp4Plan plan;
    if (!pa::plan_decode_fp4(num_seqs, num_heads, num_kv_heads, head_dim, max_seqlen_k, sliding_window, &plan))
        return 0;
    return up256(plan.workspace_bytes) +
           2 * pa::prefill_fp4_scratch_bytes(num_seqs, num_kv_heads, head_dim, max_seqlen_k);
}

size_t pa_varlen_prefill_fp4_workspace_size_q(int num_seqs, int num_heads, int num_kv_heads,
                                              int head_dim, int max_seqlen_q, int max_seqlen_k,
                                              int sliding_window) {
    if (max_seqlen_q < 0 || num_kv_heads <= 0) return 0;
    const int group = num_heads / num_kv_heads;
    if (group >= 1 && group <= 64 && pa::prefill_fp4_expands(group, max_seqlen_q))
        return pa_varlen_prefill_fp4_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_seqlen_k,
                                                    sliding_window);
    return pa_decode_fp4_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_seqlen_k, sliding_window);
}

pa_status pa_varlen_prefill_fp4(void *out, const void *q, const void *key, const void *value,
                                const int32_t *slot_mapping, void *k_cache, void *v_cache,
                                const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                const int32_t *seq_lens, const int32_t *block_table,
                                int max_num_blocks, int num_seqs, int total_q, int max_seqlen_q,
                                int max_seqlen_k, int64_t num_blocks, int block_size,
                                int num_heads, int num_kv_heads, int head_dim,
                                int sliding_window, float scale, float kv_scale, void *workspace,
                                size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || max_num_blocks < 0)
        return PA_ERR_INVALID_ARG;
    if (max_seqlen_k > kMostKeys) return PA_ERR_UNSUPPORTED;
    pa_status st = check_fp4_cache(num_blocks, block_size, num_kv_heads, head_dim, kv_scale);
    if (st == PA_OK) st = check_fp4_heads(num_heads, num_kv_heads, scale, kv_scale);
    if (st != PA_OK) return st;
    if (max_seqlen_q > max_seqlen_k) return PA_ERR_INVALID_ARG;
    if (num_seqs > 65535 || total_q > 0x7fffff00) return PA_ERR_UNSUPPORTED;
    const bool has_new = key || value || slot_mapping;
    if (has_new && !(key && value && slot_mapping)) return PA_ERR_INVALID_ARG;
    if (total_q == 0) return PA_OK;
    if (has_new) {
        if (!k_cache || !v_cache || !aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) ||
            !aligned(v_cache, 16))
            return PA_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // With no sequence there is nothing to attend, but the new tokens are still stored.
    auto store = [&]() {
        return run_store_fp4(key, value, k_cache, v_cache, slot_mapping, total_q, num_blocks, block_size,
                             num_kv_heads, head_dim, kv_scale, s);
    };
    if (num_seqs == 0) return has_new ? store() : PA_OK;
    if (!pa::prefill_fits(num_seqs, num_kv_heads, num_heads / num_kv_heads, total_q, max_seqlen_q, num_blocks * block_size))
        return PA_ERR_UNSUPPORTED;
    if (!out || !q || !k_cache || !v_cache || !block_table || !cu_seqlens_q) return PA_ERR_INVALID_ARG;
    if (!seq_lens && !cu_seqlens_k) return PA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return PA_ERR_INVALID_ARG;
    if (max_seqlen_k > 0 && max_num_blocks == 0) return PA_ERR_INVALID_ARG;
    // The workspace: what the decode kernel needs for the single-row sequences (with seq_lens),
    // then the scratch cache, if it is large enough for that too.
    pa::DecodeFp4Plan plan;
    if (!pa::plan_decode_fp4(num_seqs, num_heads, num_kv_heads, head_dim, max_seqlen_k, sliding_window, &plan))
        return PA_ERR_INVALID_ARG;
    if (seq_lens && plan.workspace_bytes > 0 && (!workspace || workspace_bytes < plan.workspace_bytes))
        return PA_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
    const size_t scratch = 2 * pa::prefill_fp4_scratch_bytes(num_seqs, num_kv_heads, head_dim, max_seqlen_k);
    const bool has_scratch = workspace && scratch > 0 && workspace_bytes >= up256(plan.workspace_bytes) + scratch;
    if (has_new) {
        st = store();
        if (st != PA_OK) return st;
    }
    pa::PrefillArgs a{};
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.cu_seqlens_q = cu_seqlens_q;
    a.cu_seqlens_k = cu_seqlens_k;
    a.seq_lens = seq_lens;
    a.block_table = block_table;
    a.max_num_blocks = max_num_blocks;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.max_seqlen_q = max_seqlen_q;
    a.max_seqlen_k = max_seqlen_k;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.sliding_window = sliding_window;
    a.scale = scale;
    a.cache = pa::kCacheFp4;
    a.kv_scale = kv_scale;
    a.workspace = workspace;
    a.scratch = has_scratch ? static_cast<uint8_t *>(workspace) + up256(plan.workspace_bytes) : nullptr;
    a.err = pa::device_error_word();
    return pa::cuda_status(pa::launch_prefill(a, s));
}

}  // extern "C"
