/*
 * pagedkv_rope.h -- the step between a layer's projections and its paged
 * cache: RMS norm of each query and key head, rotation by position, and the
 * append of K and V into their slots, in one kernel.  Part of libpagedkv.so.
 *
 * Sources (page title, section):
 *  - "Roadmap: vLLM-style serving features for TornadoVM batched decode":
 *    decode kernels with a norm of every query and key head and a rotation of
 *    split halves, run before the batched paged attention.  The page gives no
 *    formula; the two below are the usual ones.
 *  - "Distributed LLM Inference Serving Platform", section 5.1: the new
 *    token's K and V are written into the physical block assigned to it.
 *
 * For a head x of head_dim entries with weight w (NULL: no norm, y = x):
 *    y_i = x_i / sqrt(mean_j x_j^2 + eps) * w_i
 * and for a token at position p, each pair (a, b) of the first rot_dim entries
 * of y becomes
 *    (a cos_i - b sin_i, b cos_i + a sin_i),   i < rot_dim / 2,
 * with cos_i and sin_i from row p of the caller's table.  The pairs are
 * (y_i, y_{i + rot_dim/2}) or, interleaved, (y_{2i}, y_{2i+1}); the other
 * entries stay as they are.  All of it in fp32 from the fp16 inputs, rounded
 * once on the store (to fp16, or to E4M3).
 */
#ifndef PAGEDKV_ROPE_H
#define PAGEDKV_ROPE_H

#include <stddef.h>
#include <stdint.h>

#include "pagedkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bit of the device error word, beside those of pagedkv.h: a token's position
 * outside [0, max_positions). */
#define PKV_ERRBIT_POSITION 0x40

/*
 * Norm, rotation and append of num_tokens new tokens.
 *
 *  q_out          device fp16 [num_tokens][n_q_heads][head_dim], contiguous;
 *                 may be q itself where q_stride is n_q_heads * head_dim
 *  q, k, v        device fp16: token i's heads are contiguous, [heads][head_dim]
 *                 starting at element i * stride (so all three may be columns
 *                 of one fused projection's output)
 *  q_stride, k_stride, v_stride   elements from one token to the next: a
 *                 multiple of 8, at least heads * head_dim
 *  q_weight, k_weight   device fp16 [head_dim], each may be NULL (no norm of
 *                 those heads; their rotation runs all the same)
 *  eps            finite, >= 0
 *  cos_sin        device fp32 [max_positions][rot_dim]: row p holds cos_0 ..
 *                 cos_{rot_dim/2-1}, then sin_0 .. sin_{rot_dim/2-1}; NULL
 *                 when rot_dim is 0
 *  positions      device int32 [num_tokens]; NULL when rot_dim is 0
 *  rot_dim        0 (no rotation) or a multiple of 16, at most head_dim
 *  interleaved    0: pairs (i, i + rot_dim/2); 1: pairs (2i, 2i + 1)
 *  slot_mapping, k_cache, v_cache, block_size, num_blocks, err_word,
 *  cuda_stream    as for paged_kv_append
 *  head_dim       a multiple of 8, at most 256 (E4M3: of 16)
 *
 * V is copied bit for bit.  A token with a negative slot is padding: nothing
 * is written for it, its row of q_out included.  A slot beyond the pool
 * sets PKV_ERRBIT_SLOT and a position outside the table PKV_ERRBIT_POSITION;
 * that token is skipped as a whole.  Two tokens with one slot in a call: which
 * one lands is unspecified.  Pointers 16-byte aligned (positions 4,
 * slot_mapping 8).  num_tokens == 0 is a no-op.
 */
int paged_qk_norm_rope_append(void *q_out, const void *q, const void *k, const void *v,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              const void *q_weight, const void *k_weight, float eps,
                              const float *cos_sin, const int32_t *positions, int max_positions,
                              int rot_dim, int interleaved, const int64_t *slot_mapping,
                              void *k_cache, void *v_cache, int num_tokens, int n_q_heads,
                              int n_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                              int32_t *err_word, void *cuda_stream);

/*
 * The same into E4M3 caches (the format and scales of paged_kv_append_fp8):
 * K is stored as E4M3(y / k_scale) from the fp32 value of the norm and the
 * rotation, with no fp16 value in between, and V as paged_kv_append_fp8
 * stores it.  q_out stays fp16.
 */
int paged_qk_norm_rope_append_fp8(void *q_out, const void *q, const void *k, const void *v,
                                  int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                  const void *q_weight, const void *k_weight, float eps,
                                  const float *cos_sin, const int32_t *positions,
                                  int max_positions, int rot_dim, int interleaved,
                                  const int64_t *slot_mapping, void *k_cache, void *v_cache,
                                  int num_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                                  int block_size, int64_t num_blocks, float k_scale,
                                  float v_scale, int32_t *err_word, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_ROPE_H */
