// q8_api.cu -- the entry points of include/pagedkv_q8.h: argument checks on the
// host, launches on the caller's stream.  Allocates nothing.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "pagedkv_q8.h"
#include "pkv_internal.h"
#include "q8.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool stride_ok(int64_t stride, int64_t least) { return stride % 8 == 0 && stride >= least; }

int status_of(cudaError_t e) {
    if (e == cudaErrorInvalidValue) return PKV_ERR_UNSUPPORTED;
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// What every call says about its cache.
int check_cache(int kind, int n_kv_heads, int head_dim, int block_size, int64_t num_blocks) {
    if ((kind != PKV_Q8_E4M3 && kind != PKV_Q8_INT8) || n_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0)
        return PKV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32 && block_size != 64 &&
                                                block_size != 128 && block_size != 256))
        return PKV_ERR_UNSUPPORTED;
    // rows (of all heads) are numbered in 31 bits
    if (num_blocks > INT32_MAX / n_kv_heads / block_size) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

bool cache_ok(const void *k_cache, const void *v_cache, const float *k_scales, const float *v_scales) {
    return k_cache && v_cache && k_scales && v_scales && aligned(k_cache, 16) && aligned(v_cache, 16) &&
           aligned(k_scales, 4) && aligned(v_scales, 4);
}

int sm_count(int *out) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    const bool keep = dev >= 0 && dev < kMaxDevices;
    if (keep) n = cached[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return PKV_ERR_CUDA;
        if (keep) cached[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return PKV_OK;
}

struct Plan {
    int max_len;
    bool empty;  // nothing to launch
    int most, sms;  // tokens of a sequence that can be new; of the device
    pkv::Q8Split split;
};

int make_plan(int num_seqs, int total_q, int max_q_len, int n_q_heads, int n_kv_heads, int head_dim,
              int block_size, int max_blocks_per_seq, int max_context_len, Plan *plan) {
    if (num_seqs < 0 || total_q < 0 || max_q_len < 0 || n_q_heads <= 0 || n_kv_heads <= 0 ||
        max_blocks_per_seq <= 0 || n_q_heads % n_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    const int rc = check_cache(PKV_Q8_E4M3, n_kv_heads, head_dim, block_size, 1);
    if (rc != PKV_OK) return rc;
    if (num_seqs > pkv::kQ8MaxSeqs || n_q_heads / n_kv_heads > pkv::kQ8MaxGroup) return PKV_ERR_UNSUPPORTED;
    const long long cap = static_cast<long long>(max_blocks_per_seq) * block_size;
    if (cap > (1LL << 30)) return PKV_ERR_INVALID_ARG;
    if (static_cast<long long>(total_q) * n_q_heads > (1LL << 30) ||
        static_cast<long long>(max_q_len) * n_q_heads > (1LL << 30))
        return PKV_ERR_UNSUPPORTED;
    long long max_len = max_context_len <= 0 ? cap : max_context_len;
    if (max_len > cap) max_len = cap;
    plan->max_len = static_cast<int>(max_len);
    plan->empty = num_seqs == 0 || total_q == 0 || max_q_len == 0;
    plan->split.ws_bytes = 0;
    if (plan->empty) return PKV_OK;
    // no sequence has more new tokens than there are
    plan->most = max_q_len < total_q ? max_q_len : total_q;
    if (!pkv::q8_fits(num_seqs, plan->most, n_q_heads, n_kv_heads, plan->max_len)) return PKV_ERR_UNSUPPORTED;
    if (sm_count(&plan->sms) != PKV_OK) return PKV_ERR_CUDA;
    plan->split = pkv::q8_split(plan->most, n_q_heads, n_kv_heads, head_dim, plan->sms);
    return PKV_OK;
}

}  // namespace

extern "C" {

int paged_kv_append_q8(const void *k_new, const void *v_new, int64_t k_stride, int64_t v_stride,
                       const int32_t *query_start, const int32_t *block_tables,
                       const int32_t *context_lens, int num_seqs, int total, int max_q_len,
                       int max_blocks_per_seq, void *k_cache, void *v_cache, float *k_scales,
                       float *v_scales, int kind, int n_kv_heads, int head_dim, int block_size,
                       int64_t num_blocks, int32_t *err_word, void *cuda_stream) {
    const int rc = check_cache(kind, n_kv_heads, head_dim, block_size, num_blocks);
    if (rc != PKV_OK) return rc;
    if (num_seqs < 0 || total < 0 || max_q_len < 0 || max_blocks_per_seq <= 0) return PKV_ERR_INVALID_ARG;
    if (!query_start && (total != num_seqs || (num_seqs > 0 && max_q_len != 1))) return PKV_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(n_kv_heads) * head_dim;
    if (!stride_ok(k_stride, width) || !stride_ok(v_stride, width)) return PKV_ERR_INVALID_ARG;
    if (num_seqs > pkv::kQ8MaxSeqs) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total == 0 || max_q_len == 0) return PKV_OK;
    if (!k_new || !v_new || !block_tables || !context_lens || !cache_ok(k_cache, v_cache, k_scales, v_scales))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        (query_start && !aligned(query_start, 4)) || (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    pkv::Q8AppendArgs a{};
    a.k_new = k_new;
    a.v_new = v_new;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.query_start = query_start;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.num_seqs = num_seqs;
    a.total = total;
    a.max_q_len = max_q_len;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    a.err = err_word;
    return status_of(pkv::launch_q8_append(a, kind, static_cast<cudaStream_t>(cuda_stream)));
}

int paged_decode_q8_plan(int num_seqs, int total_q, int max_q_len, int n_q_heads, int n_kv_heads,
                         int head_dim, int block_size, int max_blocks_per_seq,
                         int max_context_len, size_t *workspace_bytes_out) {
    Plan plan{};
    const int rc = make_plan(num_seqs, total_q, max_q_len, n_q_heads, n_kv_heads, head_dim, block_size,
                             max_blocks_per_seq, max_context_len, &plan);
    if (rc == PKV_OK && workspace_bytes_out)
        *workspace_bytes_out = plan.empty ? 0 : pkv::q8_plan_bytes(plan.most, n_q_heads, n_kv_heads, head_dim, plan.sms);
    return rc;
}

int paged_decode_attention_q8(void *out, const void *q, int64_t q_stride, const void *k_cache,
                              const void *v_cache, const float *k_scales, const float *v_scales,
                              int kind, const int32_t *block_tables, const int32_t *context_lens,
                              const int32_t *query_start, int num_seqs, int total_q,
                              int max_q_len, int max_blocks_per_seq, int64_t num_blocks,
                              float scale, int n_q_heads, int n_kv_heads, int head_dim,
                              int block_size, int max_context_len, void *workspace,
                              size_t workspace_bytes, float *lse_out, int32_t *err_word,
                              void *cuda_stream, uint32_t flags) {
    int rc = check_cache(kind, n_kv_heads, head_dim, block_size, num_blocks);
    if (rc != PKV_OK) return rc;
    if (!std::isfinite(scale) || std::fabs(scale) >= 1e38f || (flags & ~PKV_TABLES_READY))
        return PKV_ERR_INVALID_ARG;
    if (!query_start && (total_q != num_seqs || (num_seqs > 0 && max_q_len != 1))) return PKV_ERR_INVALID_ARG;
    Plan plan{};
    rc = make_plan(num_seqs, total_q, max_q_len, n_q_heads, n_kv_heads, head_dim, block_size,
                   max_blocks_per_seq, max_context_len, &plan);
    if (rc != PKV_OK) return rc;
    if (!stride_ok(q_stride, static_cast<int64_t>(n_q_heads) * head_dim)) return PKV_ERR_INVALID_ARG;
    if (plan.empty) return PKV_OK;
    if (!out || !q || !block_tables || !context_lens || !cache_ok(k_cache, v_cache, k_scales, v_scales))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        (query_start && !aligned(query_start, 4)) || (lse_out && !aligned(lse_out, 4)) ||
        (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < plan.split.ws_bytes || !aligned(workspace, 256))
        return PKV_ERR_WORKSPACE;
    pkv::Q8AttentionArgs a{};
    a.out = out;
    a.q = q;
    a.q_stride = q_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.max_q_len = plan.most;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.max_context_len = plan.max_len;
    a.by_group = pkv::q8_divide_by(n_q_heads / n_kv_heads);
    a.record_rows = plan.split.record_rows;
    a.tile_tokens = plan.split.tile_tokens;
    a.workspace = workspace;
    a.lse_out = lse_out;
    a.err = err_word;
    a.tables_ready = (flags & PKV_TABLES_READY) ? 1 : 0;
    a.first_wait_polls = pkv::test_wait_polls();
    return status_of(pkv::launch_q8_attention(a, kind, plan.split, static_cast<cudaStream_t>(cuda_stream)));
}

int paged_kv_gather_q8(void *k, void *v, const void *k_cache, const void *v_cache,
                       const float *k_scales, const float *v_scales, int kind,
                       const int32_t *block_tables, const int32_t *start, int num_seqs,
                       int64_t total, int max_blocks_per_seq, int64_t num_blocks,
                       int n_kv_heads, int head_dim, int block_size, int32_t *err_word,
                       void *cuda_stream) {
    const int rc = check_cache(kind, n_kv_heads, head_dim, block_size, num_blocks);
    if (rc != PKV_OK) return rc;
    if (num_seqs < 0 || total < 0 || max_blocks_per_seq <= 0) return PKV_ERR_INVALID_ARG;
    if (total > INT32_MAX || num_seqs > pkv::kQ8MaxSeqs) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total == 0) return PKV_OK;
    if (!k || !v || !block_tables || !start || !cache_ok(k_cache, v_cache, k_scales, v_scales))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(block_tables, 4) || !aligned(start, 4) ||
        (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    const pkv::Q8GatherArgs a{k,     v,        k_cache, v_cache, k_scales, v_scales, block_tables,
                              start, num_seqs, total,   max_blocks_per_seq, num_blocks, n_kv_heads, head_dim,
                              block_size, err_word};
    return status_of(pkv::launch_q8_gather(a, kind, static_cast<cudaStream_t>(cuda_stream)));
}

int paged_kv_copy_blocks_q8(void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                            const int32_t *src, const int32_t *dst, const int32_t *tokens,
                            int num_copies, int n_kv_heads, int head_dim, int block_size,
                            int64_t num_blocks, int32_t *err_word, void *cuda_stream) {
    const int rc = check_cache(PKV_Q8_E4M3, n_kv_heads, head_dim, block_size, num_blocks);
    if (rc != PKV_OK) return rc;
    if (num_copies < 0) return PKV_ERR_INVALID_ARG;
    if (num_copies == 0) return PKV_OK;
    if (!src || !dst || !cache_ok(k_cache, v_cache, k_scales, v_scales) || !aligned(src, 4) || !aligned(dst, 4) ||
        (tokens && !aligned(tokens, 4)) || (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    const pkv::Q8CopyArgs a{k_cache,    v_cache,  k_scales,   v_scales,   src,      dst, tokens, num_copies,
                            n_kv_heads, head_dim, block_size, num_blocks, err_word};
    return status_of(pkv::launch_q8_copy(a, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
