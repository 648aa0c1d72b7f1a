// latent_api.cu -- the entry points of include/pagedkv_rope.h and
// include/pagedkv_latent.h: argument checks on the host, launches on the
// caller's stream.  Allocates nothing.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "pagedkv_latent.h"
#include "pagedkv_rope.h"
#include "pkv_internal.h"
#include "rope_latent.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A token stride: whole 16-byte pieces, at least `least` entries.
bool stride_ok(int64_t stride, int64_t least) { return stride % 8 == 0 && stride >= least; }

bool cache_block_ok(int bs) {
    return bs == 16 || bs == 32 || bs == 64 || bs == 128 || bs == 256;
}

bool scale_ok(float scale) {  // finite, in base 2 too
    return std::isfinite(scale) && std::fabs(scale) < 1e38f;
}

// |scale| * log2(e).  A scale of 0 becomes 1e-30: the weights are equal all the
// same, and a masked logit of -inf stays -inf.
float scale_log2_of(float scale) {
    const double s = std::fabs(static_cast<double>(scale)) * 1.4426950408889634;
    return s < 1e-30 ? 1e-30f : static_cast<float>(s);
}

int status_of(cudaError_t e) {
    if (e == cudaErrorInvalidValue) return PKV_ERR_UNSUPPORTED;
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int qk_append(void *q_out, const void *q, const void *k, const void *v, int64_t q_stride,
              int64_t k_stride, int64_t v_stride, const void *q_weight, const void *k_weight,
              float eps, const float *cos_sin, const int32_t *positions, int max_positions,
              int rot_dim, int interleaved, const int64_t *slot_mapping, void *k_cache,
              void *v_cache, int num_tokens, int n_q_heads, int n_kv_heads, int head_dim,
              int block_size, int64_t num_blocks, bool fp8, float k_scale, float v_scale,
              int32_t *err_word, void *cuda_stream) {
    if (num_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || head_dim % (fp8 ? 16 : 8) != 0 || !std::isfinite(eps) || eps < 0.f)
        return PKV_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0 || (interleaved & ~1))
        return PKV_ERR_INVALID_ARG;
    if (fp8 && (!std::isfinite(k_scale) || !std::isfinite(v_scale) || !(k_scale > 0.f) ||
                !(v_scale > 0.f)))
        return PKV_ERR_INVALID_ARG;
    if (head_dim > 256) return PKV_ERR_UNSUPPORTED;
    const int64_t qw = static_cast<int64_t>(n_q_heads) * head_dim;
    const int64_t kw = static_cast<int64_t>(n_kv_heads) * head_dim;
    if (!stride_ok(q_stride, qw) || !stride_ok(k_stride, kw) || !stride_ok(v_stride, kw))
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!q_out || !q || !k || !v || !slot_mapping || !k_cache || !v_cache)
        return PKV_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!cos_sin || !positions || max_positions <= 0 || !aligned(cos_sin, 16) ||
                        !aligned(positions, 4)))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_mapping, 8) ||
        (q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16)) ||
        (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    if (q_out == q && q_stride != qw) return PKV_ERR_INVALID_ARG;
    pkv::QkAppendArgs a{};
    a.q_out = q_out;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.max_positions = max_positions;
    a.rot_dim = rot_dim;
    a.interleaved = interleaved;
    a.slot_mapping = slot_mapping;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.num_tokens = num_tokens;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.num_slots = num_blocks * block_size;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.err = err_word;
    return status_of(pkv::launch_qk_append(a, fp8, static_cast<cudaStream_t>(cuda_stream)));
}

// SMs of the current device, looked up once per device.
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

struct LatentPlan {
    int max_len;
    bool empty;  // nothing to launch
    pkv::LatentSplit split;
};

int make_latent_plan(int num_seqs, int total_q, int max_q_len, int n_q_heads, int latent_dim,
                     int rope_dim, int block_size, int max_blocks_per_seq, int max_context_len,
                     LatentPlan *plan) {
    if (num_seqs < 0 || total_q < 0 || max_q_len < 0 || n_q_heads <= 0 || latent_dim <= 0 ||
        rope_dim <= 0 || max_blocks_per_seq <= 0)
        return PKV_ERR_INVALID_ARG;
    if ((latent_dim != 256 && latent_dim != 512) || rope_dim != 64 || !cache_block_ok(block_size) ||
        num_seqs > 4096)
        return PKV_ERR_UNSUPPORTED;
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
    int sms = 0;
    if (sm_count(&sms) != PKV_OK) return PKV_ERR_CUDA;
    if (!pkv::latent_split(num_seqs, max_q_len, n_q_heads, latent_dim, plan->max_len, sms,
                           &plan->split))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

}  // namespace

extern "C" {

int paged_qk_norm_rope_append(void *q_out, const void *q, const void *k, const void *v,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              const void *q_weight, const void *k_weight, float eps,
                              const float *cos_sin, const int32_t *positions, int max_positions,
                              int rot_dim, int interleaved, const int64_t *slot_mapping,
                              void *k_cache, void *v_cache, int num_tokens, int n_q_heads,
                              int n_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                              int32_t *err_word, void *cuda_stream) {
    return qk_append(q_out, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps,
                     cos_sin, positions, max_positions, rot_dim, interleaved, slot_mapping,
                     k_cache, v_cache, num_tokens, n_q_heads, n_kv_heads, head_dim, block_size,
                     num_blocks, false, 1.f, 1.f, err_word, cuda_stream);
}

int paged_qk_norm_rope_append_fp8(void *q_out, const void *q, const void *k, const void *v,
                                  int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                  const void *q_weight, const void *k_weight, float eps,
                                  const float *cos_sin, const int32_t *positions,
                                  int max_positions, int rot_dim, int interleaved,
                                  const int64_t *slot_mapping, void *k_cache, void *v_cache,
                                  int num_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                                  int block_size, int64_t num_blocks, float k_scale,
                                  float v_scale, int32_t *err_word, void *cuda_stream) {
    return qk_append(q_out, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps,
                     cos_sin, positions, max_positions, rot_dim, interleaved, slot_mapping,
                     k_cache, v_cache, num_tokens, n_q_heads, n_kv_heads, head_dim, block_size,
                     num_blocks, true, k_scale, v_scale, err_word, cuda_stream);
}

int paged_latent_append(const void *kv, int64_t kv_stride, const void *weight, float eps,
                        const float *cos_sin, const int32_t *positions, int max_positions,
                        int interleaved, const int64_t *slot_mapping, void *cache,
                        const void *q_rope, int64_t q_token_stride, int64_t q_head_stride,
                        void *q_out, int64_t out_token_stride, int64_t out_head_stride,
                        int n_q_heads, int num_tokens, int latent_dim, int rope_dim,
                        int block_size, int64_t num_blocks, int32_t *err_word,
                        void *cuda_stream) {
    if (num_tokens < 0 || latent_dim <= 0 || latent_dim % 8 != 0 || rope_dim <= 0 ||
        rope_dim % 16 != 0 || block_size <= 0 || num_blocks <= 0 || n_q_heads < 0 ||
        !std::isfinite(eps) || eps < 0.f || (interleaved & ~1) || max_positions <= 0)
        return PKV_ERR_INVALID_ARG;
    if (latent_dim > 1024 || rope_dim > 256) return PKV_ERR_UNSUPPORTED;
    if (!stride_ok(kv_stride, latent_dim + rope_dim)) return PKV_ERR_INVALID_ARG;
    const bool queries = q_rope || q_out;
    if (queries) {
        if (!q_rope || !q_out || n_q_heads <= 0) return PKV_ERR_INVALID_ARG;
        if (!stride_ok(q_head_stride, rope_dim) || !stride_ok(out_head_stride, rope_dim))
            return PKV_ERR_INVALID_ARG;
        const int64_t heads = n_q_heads - 1;
        if (!stride_ok(q_token_stride, heads * q_head_stride + rope_dim) ||
            !stride_ok(out_token_stride, heads * out_head_stride + rope_dim))
            return PKV_ERR_INVALID_ARG;
        if (q_rope == q_out &&
            (q_token_stride != out_token_stride || q_head_stride != out_head_stride))
            return PKV_ERR_INVALID_ARG;
    }
    if (num_tokens == 0) return PKV_OK;
    if (!kv || !cos_sin || !positions || !slot_mapping || !cache) return PKV_ERR_INVALID_ARG;
    if (!aligned(kv, 16) || !aligned(cos_sin, 16) || !aligned(positions, 4) ||
        !aligned(slot_mapping, 8) || !aligned(cache, 16) || (weight && !aligned(weight, 16)) ||
        (queries && (!aligned(q_rope, 16) || !aligned(q_out, 16))) ||
        (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    pkv::LatentAppendArgs a{};
    a.kv = kv;
    a.kv_stride = kv_stride;
    a.weight = weight;
    a.eps = eps;
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.max_positions = max_positions;
    a.interleaved = interleaved;
    a.slot_mapping = slot_mapping;
    a.cache = cache;
    a.q_rope = q_rope;
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.q_out = q_out;
    a.out_token_stride = out_token_stride;
    a.out_head_stride = out_head_stride;
    a.n_q_heads = queries ? n_q_heads : 0;
    a.num_tokens = num_tokens;
    a.latent_dim = latent_dim;
    a.rope_dim = rope_dim;
    a.num_slots = num_blocks * block_size;
    a.err = err_word;
    return status_of(pkv::launch_latent_append(a, static_cast<cudaStream_t>(cuda_stream)));
}

int paged_latent_plan(int num_seqs, int total_q, int max_q_len, int n_q_heads, int latent_dim,
                      int rope_dim, int block_size, int max_blocks_per_seq, int max_context_len,
                      size_t *workspace_bytes_out) {
    LatentPlan plan{};
    const int rc = make_latent_plan(num_seqs, total_q, max_q_len, n_q_heads, latent_dim, rope_dim,
                                    block_size, max_blocks_per_seq, max_context_len, &plan);
    if (rc == PKV_OK && workspace_bytes_out) *workspace_bytes_out = plan.split.ws_bytes;
    return rc;
}

int paged_latent_attention(void *out, const void *q, const void *cache,
                           const int32_t *block_tables, const int32_t *context_lens,
                           const int32_t *query_start, int num_seqs, int total_q, int max_q_len,
                           int max_blocks_per_seq, int64_t num_blocks, float scale, int n_q_heads,
                           int latent_dim, int rope_dim, int block_size, int max_context_len,
                           void *workspace, size_t workspace_bytes, float *lse_out,
                           int32_t *err_word, void *cuda_stream) {
    if (num_blocks <= 0 || !scale_ok(scale)) return PKV_ERR_INVALID_ARG;
    if (!query_start && (total_q != num_seqs || (num_seqs > 0 && max_q_len != 1)))
        return PKV_ERR_INVALID_ARG;
    if (block_size > 0 && num_blocks > INT32_MAX / block_size)  // rows are numbered in 32 bits
        return PKV_ERR_UNSUPPORTED;
    LatentPlan plan{};
    const int rc = make_latent_plan(num_seqs, total_q, max_q_len, n_q_heads, latent_dim, rope_dim,
                                    block_size, max_blocks_per_seq, max_context_len, &plan);
    if (rc != PKV_OK) return rc;
    if (plan.empty) return PKV_OK;
    if (!out || !q || !cache || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(cache, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || (query_start && !aligned(query_start, 4)) ||
        (lse_out && !aligned(lse_out, 4)) || (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < plan.split.ws_bytes || !aligned(workspace, 256))
        return PKV_ERR_WORKSPACE;
    pkv::LatentAttentionArgs a{};
    a.out = out;
    a.q = q;
    a.cache = cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.max_q_len = max_q_len;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale_log2_of(scale);
    a.negate = scale < 0.f;
    a.n_q_heads = n_q_heads;
    a.latent_dim = latent_dim;
    a.rope_dim = rope_dim;
    a.block_size = block_size;
    a.max_context_len = plan.max_len;
    a.workspace = workspace;
    a.lse_out = lse_out;
    a.err = err_word;
    a.first_wait_polls = pkv::test_wait_polls();
    return status_of(pkv::launch_latent_attention(a, plan.split, static_cast<cudaStream_t>(cuda_stream)));
}

int paged_latent_gather(void *latents, void *ropes, const void *cache,
                        const int32_t *block_tables, const int32_t *start, int num_seqs,
                        int64_t total, int max_blocks_per_seq, int64_t num_blocks,
                        int latent_dim, int rope_dim, int block_size, int32_t *err_word,
                        void *cuda_stream) {
    if (num_seqs < 0 || total < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        latent_dim <= 0 || rope_dim <= 0 || latent_dim % 8 != 0 || rope_dim % 8 != 0 ||
        block_size <= 0)
        return PKV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(latent_dim) + rope_dim > 2048 || total > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total == 0) return PKV_OK;
    if (!latents || !ropes || !cache || !block_tables || !start) return PKV_ERR_INVALID_ARG;
    if (!aligned(latents, 16) || !aligned(ropes, 16) || !aligned(cache, 16) ||
        !aligned(block_tables, 4) || !aligned(start, 4) || (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    pkv::LatentGatherArgs a{latents,  ropes, cache, block_tables, start, num_seqs, total,
                            max_blocks_per_seq, num_blocks, latent_dim, rope_dim, block_size,
                            err_word};
    return status_of(pkv::launch_latent_gather(a, static_cast<cudaStream_t>(cuda_stream)));
}

int latent_prefill_attention(void *out, const void *q, const void *kv, const void *k_rope,
                             const int32_t *q_start, const int32_t *kv_start, int num_seqs,
                             int total_q, int total_kv, int max_q_len, int max_kv_len,
                             float scale, int n_heads, int head_dim, int rope_dim,
                             float *lse_out, int32_t *err_word, void *cuda_stream) {
    if (num_seqs < 0 || total_q < 0 || total_kv < 0 || max_q_len < 0 || max_kv_len < 0 ||
        n_heads <= 0 || head_dim <= 0 || rope_dim <= 0 || !scale_ok(scale))
        return PKV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || rope_dim != 64 || n_heads > 65535 ||
        num_seqs > 65535)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PKV_OK;
    if (!out || !q || !q_start || !kv_start) return PKV_ERR_INVALID_ARG;
    // an empty tensor has no address; none of its rows is ever copied
    if (total_kv == 0) kv = k_rope = q;
    if (!kv || !k_rope) return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(kv, 16) || !aligned(k_rope, 16) ||
        !aligned(q_start, 4) || !aligned(kv_start, 4) || (lse_out && !aligned(lse_out, 4)) ||
        (err_word && !aligned(err_word, 4)))
        return PKV_ERR_INVALID_ARG;
    pkv::LatentPrefillArgs a{};
    a.out = out;
    a.q = q;
    a.kv = kv;
    a.k_rope = k_rope;
    a.q_start = q_start;
    a.kv_start = kv_start;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.total_kv = total_kv;
    a.max_q_len = max_q_len < total_q ? max_q_len : total_q;  // CTAs for no more rows than there are
    a.max_kv_len = max_kv_len;
    a.scale_log2 = scale_log2_of(scale);
    a.negate = scale < 0.f;
    a.n_heads = n_heads;
    a.head_dim = head_dim;
    a.rope_dim = rope_dim;
    a.lse_out = lse_out;
    a.err = err_word;
    a.first_wait_polls = pkv::test_wait_polls();
    int sms = 0;
    if (sm_count(&sms) != PKV_OK) return PKV_ERR_CUDA;
    return status_of(pkv::launch_latent_prefill(a, sms, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
