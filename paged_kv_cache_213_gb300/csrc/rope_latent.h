// rope_latent.h -- launch interfaces of the norm/rotation append and of the
// latent attention kernels (rope_append.cu, latent_*.cu).  Not public.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace pkv {

// Lets a kernel have `bytes` of dynamic shared memory on the current device, once a
// device (`done`: a bit per device, one variable a kernel).
template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t a = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (a == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return a;
}

struct QkAppendArgs {
    void *q_out;
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const void *q_weight, *k_weight;
    float eps;
    const float *cos_sin;
    const int32_t *positions;
    int max_positions, rot_dim, interleaved;
    const int64_t *slot_mapping;
    void *k_cache, *v_cache;
    int num_tokens, n_q_heads, n_kv_heads, head_dim, block_size;
    long long num_slots;
    float k_scale, v_scale;
    int32_t *err;
    // set by the launcher: lanes per head, warps per token, those for queries and for
    // keys (or values)
    int width_log2, jobs, q_jobs, kv_jobs;
    float inv_dim, k_inv, v_inv;  // 1 / head_dim; 1 / scale, or 0: divide instead
};
// cudaErrorInvalidValue: more (token, head) pairs than the grid's 32-bit index.
cudaError_t launch_qk_append(QkAppendArgs a, bool fp8, cudaStream_t stream);

struct LatentAppendArgs {
    const void *kv;
    long long kv_stride;
    const void *weight;
    float eps;
    const float *cos_sin;
    const int32_t *positions;
    int max_positions, interleaved;
    const int64_t *slot_mapping;
    void *cache;
    const void *q_rope;
    long long q_token_stride, q_head_stride;
    void *q_out;
    long long out_token_stride, out_head_stride;
    int n_q_heads;  // 0: no queries
    int num_tokens, latent_dim, rope_dim;
    long long num_slots;
    int32_t *err;
    int width_log2, jobs;  // lanes per query head, warps per token: set by the launcher
};
cudaError_t launch_latent_append(LatentAppendArgs a, cudaStream_t stream);

struct LatentGatherArgs {
    void *latents, *ropes;
    const void *cache;
    const int32_t *block_tables, *start;
    int num_seqs;
    long long total;
    int max_blocks_per_seq;
    long long num_blocks;
    int latent_dim, rope_dim, block_size;
    int32_t *err;
};
cudaError_t launch_latent_gather(const LatentGatherArgs &a, cudaStream_t stream);

struct LatentAttentionArgs {
    void *out;
    const void *q, *cache;
    const int32_t *block_tables, *context_lens, *query_start;
    int num_seqs, total_q, max_q_len, max_blocks_per_seq;
    long long num_blocks;
    float scale_log2;  // |scale| * log2(e), at least 1e-30: a masked logit stays -inf
    int negate;        // the scale is negative
    int n_q_heads, latent_dim, rope_dim, block_size, max_context_len;
    void *workspace;
    float *lse_out;
    int32_t *err;
    int first_wait_polls;  // test hook, as in DecodeArgs: the first wait for a tile
};
// How a call's work is split: `workers` of `ctas` CTAs with `rows`
// query rows each, one CTA per SM.
struct LatentSplit {
    int rows, ctas, workers;
    int by_segment;  // the join's records: one per segment (sequence and row tile), else one per worker
    int records;
    int join_threads;
    size_t ws_bytes;
};
// false: more than 2^31 units of work.
bool latent_split(int num_seqs, int max_q_len, int heads, int latent_dim, int max_len, int sms,
                  LatentSplit *sp);
cudaError_t launch_latent_attention(const LatentAttentionArgs &a, const LatentSplit &sp,
                                    cudaStream_t stream);

struct LatentPrefillArgs {
    void *out;
    const void *q, *kv, *k_rope;
    const int32_t *q_start, *kv_start;
    int num_seqs, total_q, total_kv, max_q_len, max_kv_len;
    float scale_log2;  // |scale| * log2(e), at least 1e-30: a masked logit stays -inf
    int negate;        // the scale is negative
    int n_heads, head_dim, rope_dim;
    float *lse_out;
    int32_t *err;
    int first_wait_polls;  // test hook, as in DecodeArgs: the first wait for keys
};
cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int sms, cudaStream_t stream);

}  // namespace pkv
