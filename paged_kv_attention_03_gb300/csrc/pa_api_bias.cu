// pa_api_bias.cu - the extern "C" boundary of attention on packed plain rows, its gradient, and of
// the learned relative position bias (packed, decode and prefill over the paged cache).  Host-side
// argument validation only.
#include <cuda_runtime.h>

#include "pa_gb300.h"
#include "pa_internal.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

// A bias, given by table, number of buckets and largest distance: all or nothing.
pa_status check_bias(const float *bias, int num_buckets, int max_distance, float scale, pa::RelativeBias *b) {
    if (bias == nullptr) return num_buckets == 0 ? PA_OK : PA_ERR_INVALID_ARG;
    if (num_buckets < 2 || max_distance <= num_buckets / 2 || !aligned(bias, 4)) return PA_ERR_INVALID_ARG;
    if (scale < 1e-20f) return PA_ERR_UNSUPPORTED;  // (biases are divided by it)
    if (!pa::plan_relative_bias(num_buckets, max_distance, b)) return PA_ERR_UNSUPPORTED;
    b->bias = bias;
    return PA_OK;
}

pa_status check_heads(int num_heads, int num_kv_heads, int head_dim, float scale) {
    if (num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < 1.0e38f)) return PA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_heads / num_kv_heads > 64) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// Rows of `heads` heads, `stride` elements apart.
bool row_stride_ok(int64_t stride, int heads, int head_dim) {
    return stride >= static_cast<int64_t>(heads) * head_dim && stride % 8 == 0 && stride < (1ll << 38);
}

bool packed_sizes_ok(int total_q, int total_k, int num_seqs) {
    return total_q < (1 << 30) && total_k < (1 << 30) && num_seqs <= 65535;
}

// What both directions of packed attention check.  PA_OK with *nothing set: no row to compute.
pa_status check_packed(const pa::PackedArgs &a, bool *nothing) {
    if (a.num_seqs < 0 || a.total_q < 0 || a.total_k < 0 || a.max_seqlen_q < 0 || a.max_seqlen_k < 0) return PA_ERR_INVALID_ARG;
    const pa_status st = check_heads(a.num_heads, a.num_kv_heads, a.head_dim, a.scale);
    if (st != PA_OK) return st;
    if (!row_stride_ok(a.q_stride, a.num_heads, a.head_dim) || !row_stride_ok(a.k_stride, a.num_kv_heads, a.head_dim) ||
        !row_stride_ok(a.v_stride, a.num_kv_heads, a.head_dim))
        return PA_ERR_INVALID_ARG;
    if (!packed_sizes_ok(a.total_q, a.total_k, a.num_seqs)) return PA_ERR_UNSUPPORTED;
    // The kernels count tiles of at least two tokens (queries) or 128 rows in 32 bits.
    const int64_t tiles_q = (static_cast<int64_t>(a.max_seqlen_q) + 127) / 128 * a.num_seqs * a.num_heads;
    const int64_t tiles_k = (static_cast<int64_t>(a.max_seqlen_k) + 127) / 128 * a.num_seqs * a.num_kv_heads;
    if (tiles_q > 0x7fffffffLL || tiles_k > 0x7fffffffLL || a.max_seqlen_q > (1 << 30) || a.max_seqlen_k > (1 << 30) ||
        (a.num_seqs > 0 && !pa::prefill_fits(a.num_seqs, a.num_kv_heads, a.num_heads / a.num_kv_heads, a.total_q,
                                             a.max_seqlen_q > 0 ? a.max_seqlen_q : 1, a.total_k)))
        return PA_ERR_UNSUPPORTED;
    *nothing = a.num_seqs == 0 || (a.total_q == 0 && a.total_k == 0);
    if (*nothing) return PA_OK;
    if (!a.cu_seqlens_q || !a.cu_seqlens_k) return PA_ERR_INVALID_ARG;
    if (a.total_q > 0 && (!a.q || !aligned(a.q, 16))) return PA_ERR_INVALID_ARG;
    if (a.total_k > 0 && (!a.k || !a.v || !aligned(a.k, 16) || !aligned(a.v, 16))) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

}  // namespace

extern "C" {

size_t pa_relative_bias_workspace_size(int num_heads, int num_buckets, int max_distance) {
    pa::RelativeBias b{};
    if (num_heads <= 0 || !pa::plan_relative_bias(num_buckets, max_distance, &b)) return 0;
    return pa::bias_table_bytes(num_heads, b);
}

size_t pa_varlen_attn_backward_workspace_size(int total_q, int total_k, int num_seqs, int num_heads, int num_buckets,
                                              int max_distance) {
    if (total_q < 0 || total_k < 0 || num_seqs < 0 || num_heads <= 0 || !packed_sizes_ok(total_q, total_k, num_seqs)) return 0;
    pa::RelativeBias b{};
    if (num_buckets != 0 && !pa::plan_relative_bias(num_buckets, max_distance, &b)) return 0;
    size_t bytes = 0;
    if (!pa::packed_grad_workspace(total_q, total_k, num_seqs, num_heads, num_buckets, &bytes)) return 0;
    return bytes + (num_buckets > 0 ? pa::bias_table_bytes(num_heads, b) : 0);
}

pa_status pa_varlen_attn(void *out, float *lse, const void *q, const void *k, const void *v, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                         int num_seqs, int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int num_heads,
                         int num_kv_heads, int head_dim, int sliding_window, float scale, const float *bias,
                         int num_buckets, int max_distance, void *workspace, size_t workspace_bytes, void *stream) {
    pa::PackedArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.cu_seqlens_q = cu_seqlens_q;
    a.cu_seqlens_k = cu_seqlens_k;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.total_k = total_k;
    a.max_seqlen_q = max_seqlen_q;
    a.max_seqlen_k = max_seqlen_k;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.sliding_window = sliding_window < max_seqlen_k ? sliding_window : 0;  // (a window that hides nothing)
    a.scale = scale;
    bool nothing = false;
    pa_status st = check_packed(a, &nothing);
    if (st == PA_OK) st = check_bias(bias, num_buckets, max_distance, scale, &a.bias);
    if (st != PA_OK || nothing || total_q == 0) return st;
    if (!out || !lse || !aligned(out, 16) || !aligned(lse, 4)) return PA_ERR_INVALID_ARG;
    const size_t need = bias ? pa::bias_table_bytes(num_heads, a.bias) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return PA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.err = pa::device_error_word();
    if (bias) {
        a.bias_table = static_cast<float *>(workspace);
        st = pa::cuda_status(pa::launch_bias_table(static_cast<float *>(workspace), num_heads, a.bias, s));
        if (st != PA_OK) return st;
    }
    return pa::cuda_status(pa::launch_packed_attn(a, out, lse, s));
}

pa_status pa_varlen_attn_backward(void *dq, void *dk, void *dv, float *dbias, int64_t dq_stride, int64_t dk_stride,
                                  int64_t dv_stride, const void *dout, const void *q, const void *k, const void *v,
                                  const void *out, const float *lse, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                  const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int num_seqs, int total_q,
                                  int total_k, int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                                  int head_dim, int sliding_window, float scale, const float *bias, int num_buckets,
                                  int max_distance, void *workspace, size_t workspace_bytes, void *stream) {
    pa::PackedGradArgs g{};
    pa::PackedArgs &a = g.fwd;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.cu_seqlens_q = cu_seqlens_q;
    a.cu_seqlens_k = cu_seqlens_k;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.total_k = total_k;
    a.max_seqlen_q = max_seqlen_q;
    a.max_seqlen_k = max_seqlen_k;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.sliding_window = sliding_window < max_seqlen_k ? sliding_window : 0;
    a.scale = scale;
    bool nothing = false;
    pa_status st = check_packed(a, &nothing);
    if (st == PA_OK) st = check_bias(bias, num_buckets, max_distance, scale, &a.bias);
    if (st != PA_OK) return st;
    if (!row_stride_ok(dq_stride, num_heads, head_dim) || !row_stride_ok(dk_stride, num_kv_heads, head_dim) ||
        !row_stride_ok(dv_stride, num_kv_heads, head_dim))
        return PA_ERR_INVALID_ARG;
    if ((bias != nullptr) != (dbias != nullptr) || !aligned(dbias, 4)) return PA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (nothing) {  // no pair of a query and a key: the bias has no gradient
        return dbias ? pa::cuda_status(cudaMemsetAsync(dbias, 0, sizeof(float) * num_buckets * num_heads, s)) : PA_OK;
    }
    if (total_q > 0 && (!dq || !out || !lse || !dout || !aligned(dq, 16) || !aligned(out, 16) || !aligned(dout, 16) || !aligned(lse, 4)))
        return PA_ERR_INVALID_ARG;
    if (total_k > 0 && (!dk || !dv || !aligned(dk, 16) || !aligned(dv, 16))) return PA_ERR_INVALID_ARG;
    size_t need = 0;
    if (!pa::packed_grad_workspace(total_q, total_k, num_seqs, num_heads, num_buckets, &need)) return PA_ERR_UNSUPPORTED;
    const size_t table = bias ? pa::bias_table_bytes(num_heads, a.bias) : 0;
    if (need + table > 0 && (!workspace || workspace_bytes < need + table || !aligned(workspace, 256))) return PA_ERR_INVALID_ARG;
    a.err = pa::device_error_word();
    if (bias) a.bias_table = static_cast<float *>(workspace);
    g.out = out;
    g.dout = dout;
    g.lse = lse;
    g.dq = dq;
    g.dk = dk;
    g.dv = dv;
    g.dq_stride = dq_stride;
    g.dk_stride = dk_stride;
    g.dv_stride = dv_stride;
    g.dbias = dbias;
    g.workspace = static_cast<uint8_t *>(workspace) + table;
    return pa::cuda_status(pa::launch_packed_attn_backward(g, s));
}

pa_status pa_decode_bias(void *out, const void *q, const void *key, const void *value, const int32_t *slot_mapping,
                         void *k_cache, void *v_cache, const int32_t *block_table, int max_num_blocks,
                         const int32_t *seq_lens, int batch, int max_seq_len, int64_t num_blocks, int block_size,
                         int num_heads, int num_kv_heads, int head_dim, int sliding_window, float scale,
                         const float *bias, int num_buckets, int max_distance, int num_splits, void *workspace,
                         size_t workspace_bytes, void *stream) {
    if (batch < 0 || max_seq_len < 0 || num_blocks < 0 || max_num_blocks < 0 || block_size <= 0) return PA_ERR_INVALID_ARG;
    pa_status st = check_heads(num_heads, num_kv_heads, head_dim, scale);
    if (st != PA_OK) return st;
    if (!is_pow2(block_size) || block_size > 1024 || batch > 65535) return PA_ERR_UNSUPPORTED;
    pa::DecodeArgs a{};
    if (!bias) return PA_ERR_INVALID_ARG;
    st = check_bias(bias, num_buckets, max_distance, scale, &a.bias);
    if (st != PA_OK) return st;
    const bool has_new = key || value || slot_mapping;
    if (has_new && !(key && value && slot_mapping)) return PA_ERR_INVALID_ARG;
    if (batch == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_table || !seq_lens) return PA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        (has_new && (!aligned(key, 16) || !aligned(value, 16))))
        return PA_ERR_INVALID_ARG;
    if (max_seq_len > 0 && max_num_blocks == 0) return PA_ERR_INVALID_ARG;
    pa::DecodePlan plan;
    if (!pa::plan_decode(batch, num_heads, num_kv_heads, head_dim, max_seq_len, sliding_window, num_splits, &plan))
        return PA_ERR_INVALID_ARG;
    const size_t need = pa::decode_workspace_bytes(batch, num_heads, head_dim, plan);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return PA_ERR_INVALID_ARG;
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
    a.workspace = workspace;
    a.key = key;
    a.value = value;
    a.slot_mapping = slot_mapping;
    a.k_cache_w = k_cache;
    a.v_cache_w = v_cache;
    a.err = pa::device_error_word();
    return pa::cuda_status(pa::launch_decode(a, plan, static_cast<cudaStream_t>(stream)));
}

pa_status pa_varlen_prefill_bias(void *out, const void *q, const void *key, const void *value, const int32_t *slot_mapping,
                                 void *k_cache, void *v_cache, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                 const int32_t *seq_lens, const int32_t *block_table, int max_num_blocks, int num_seqs,
                                 int total_q, int max_seqlen_q, int max_seqlen_k, int64_t num_blocks, int block_size,
                                 int num_heads, int num_kv_heads, int head_dim, int sliding_window, float scale,
                                 const float *bias, int num_buckets, int max_distance, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || max_num_blocks < 0 || num_blocks < 0 || block_size <= 0)
        return PA_ERR_INVALID_ARG;
    pa_status st = check_heads(num_heads, num_kv_heads, head_dim, scale);
    if (st != PA_OK) return st;
    if (!is_pow2(block_size) || block_size < 16 || block_size > 256) return PA_ERR_UNSUPPORTED;
    if (max_seqlen_q > max_seqlen_k) return PA_ERR_INVALID_ARG;
    if (num_seqs > 65535 || total_q > 0x7fffff00 || num_blocks * block_size > 0x7fffff00LL) return PA_ERR_UNSUPPORTED;
    pa::PrefillArgs a{};
    if (!bias) return PA_ERR_INVALID_ARG;
    st = check_bias(bias, num_buckets, max_distance, scale, &a.bias);
    if (st != PA_OK) return st;
    const bool has_new = key || value || slot_mapping;
    if (has_new && !(key && value && slot_mapping)) return PA_ERR_INVALID_ARG;
    if (total_q == 0) return PA_OK;
    if (has_new && (!k_cache || !v_cache || !aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16)))
        return PA_ERR_INVALID_ARG;
    const size_t need = pa::bias_table_bytes(num_heads, a.bias);
    if (num_seqs > 0) {
        if (!pa::prefill_fits(num_seqs, num_kv_heads, num_heads / num_kv_heads, total_q, max_seqlen_q, num_blocks * block_size))
            return PA_ERR_UNSUPPORTED;
        if (!out || !q || !k_cache || !v_cache || !block_table || !cu_seqlens_q) return PA_ERR_INVALID_ARG;
        if (!seq_lens && !cu_seqlens_k) return PA_ERR_INVALID_ARG;
        if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return PA_ERR_INVALID_ARG;
        if (max_seqlen_k > 0 && max_num_blocks == 0) return PA_ERR_INVALID_ARG;
        if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (has_new) {
        st = pa_store_kvcache(key, value, k_cache, v_cache, slot_mapping, total_q, num_blocks, block_size, num_kv_heads, head_dim,
                              stream);
        if (st != PA_OK) return st;
    }
    if (num_seqs == 0 || max_seqlen_q == 0) return PA_OK;
    // (The table serves the prefill kernel; single-row sequences alone go to the decode kernel.)
    if (!seq_lens || max_seqlen_q > 1) {
        st = pa::cuda_status(pa::launch_bias_table(static_cast<float *>(workspace), num_heads, a.bias, s));
        if (st != PA_OK) return st;
    }
    a.bias_table = static_cast<float *>(workspace);
    a.bias_last = a.bias.last();
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
    a.err = pa::device_error_word();
    return pa::cuda_status(pa::launch_prefill(a, s));
}

}  // extern "C"
