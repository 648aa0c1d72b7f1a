// q8.h -- launch interfaces of the 8-bit caches with block scales
// (include/pagedkv_q8.h), between q8_api.cu and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "pagedkv_q8.h"

namespace pkv {

constexpr int kQ8MaxSeqs = 2048, kQ8MaxGroup = 128;  // a tile has 128 rows

struct Q8AppendArgs {
    const void *k_new, *v_new;
    long long k_stride, v_stride;  // elements between tokens
    const int32_t *query_start;    // NULL: token b is sequence b's
    const int32_t *block_tables, *context_lens;
    int num_seqs, total, max_q_len, max_blocks_per_seq;
    void *k_cache, *v_cache;
    float *k_scales, *v_scales;
    int n_kv_heads, head_dim, block_size;
    long long num_blocks;
    int32_t *err;
};
cudaError_t launch_q8_append(const Q8AppendArgs &a, int kind, cudaStream_t stream);

struct Q8GatherArgs {
    void *k, *v;
    const void *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    const int32_t *block_tables, *start;
    int num_seqs;
    long long total;
    int max_blocks_per_seq;
    long long num_blocks;
    int n_kv_heads, head_dim, block_size;
    int32_t *err;
};
cudaError_t launch_q8_gather(const Q8GatherArgs &a, int kind, cudaStream_t stream);

struct Q8CopyArgs {
    void *k_cache, *v_cache;
    float *k_scales, *v_scales;
    const int32_t *src, *dst, *tokens;
    int num_copies, n_kv_heads, head_dim, block_size;
    long long num_blocks;
    int32_t *err;
};
cudaError_t launch_q8_copy(const Q8CopyArgs &a, cudaStream_t stream);

// Division of x < 2^31 by d as a product: with 2^(s - 1) < d <= 2^s and mul = ceil(2^(31 + s)
// / d) = (2^(31 + s) + e) / d, 0 <= e < d, x * mul / 2^(31 + s) = x / d + x e / (d 2^(31 + s)),
// and the last term is below 1 / d, too little to reach the next whole number.
struct Q8Divide {
    uint32_t mul;
    int shift;
};
inline Q8Divide q8_divide_by(uint32_t d) {
    int s = 0;
    while ((1ull << s) < d) ++s;
    return Q8Divide{static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

struct Q8AttentionArgs {
    void *out;
    const void *q;
    long long q_stride;  // elements between tokens
    const void *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    const int32_t *block_tables, *context_lens, *query_start;
    int num_seqs, total_q, max_q_len, max_blocks_per_seq;
    long long num_blocks;
    float scale_log2;  // scale * log2(e), either sign
    int n_q_heads, n_kv_heads, head_dim, block_size, max_context_len;
    Q8Divide by_group;  // query heads of a KV head
    int record_rows, tile_tokens;  // of Q8Split
    void *workspace;
    float *lse_out;
    int32_t *err;
    int tables_ready;  // the kernel before writes no lengths, tables or query starts
    int first_wait_polls;  // test hook, as in DecodeArgs
};
// How a call's work is split: `ctas` CTAs of the kernel for `row_tiles` x 8 query rows.
struct Q8Split {
    int row_tiles;  // 0: the kernel of q8_prefill.cu
    int ctas;
    int record_rows;  // query rows that a segment has at most
    int tile_tokens;  // of q8_prefill.cu: tokens of a tile of 128 rows
    size_t ws_bytes;
};
// Units of work that a call may have: they are counted in ints, some thousands ahead.
constexpr double kQ8MaxUnits = 2147483648.0 - 65536.0;
bool q8_fits(int num_seqs, int max_q_len, int n_q_heads, int n_kv_heads, int max_len);
bool q8_prefill_fits(int num_seqs, int max_q_len, int n_q_heads, int n_kv_heads, int max_len);
// Of sizes that fit.
Q8Split q8_split(int max_q_len, int n_q_heads, int n_kv_heads, int head_dim, int sms);
Q8Split q8_prefill_split(int max_q_len, int n_q_heads, int n_kv_heads, int head_dim, int sms);
// Workspace bytes that are enough for calls of these sizes and of smaller ones.
size_t q8_plan_bytes(int max_q_len, int n_q_heads, int n_kv_heads, int head_dim, int sms);
cudaError_t launch_q8_prefill(const Q8AttentionArgs &a, int kind, const Q8Split &sp,
                              cudaStream_t stream);
cudaError_t launch_q8_attention(const Q8AttentionArgs &a, int kind, const Q8Split &sp,
                                cudaStream_t stream);

}  // namespace pkv
