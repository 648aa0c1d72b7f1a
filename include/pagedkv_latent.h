/*
 * pagedkv_latent.h -- latent attention over a paged cache: every token keeps
 * one latent vector, shared by all heads, and one rotated key part, instead of
 * keys and values of each head.  Part of libpagedkv.so.
 *
 * Source: "Distributed LLM Inference Serving Platform", case studies: keys and
 * values compressed into one latent vector a token.  The page gives the idea
 * and the saving only; the formulas are the usual ones of this attention:
 *
 *   token t:  latent c_t [latent_dim], rotated key part r_t [rope_dim]
 *   head h:   k_{t,h} = [W^K_h c_t, r_t],   v_{t,h} = W^V_h c_t
 *   logits    scale * (q^n_h . W^K_h c_t + q^r_h . r_t)
 *
 * Expanded form (prompts): the caller multiplies the latents by [W^K_h, W^V_h]
 * and latent_prefill_attention attends over these keys and values.  Absorbed
 * form (decode): with q'_h = (W^K_h)^T q^n_h the logits are scale * ([q'_h,
 * q^r_h] . [c_t, r_t]) and the output is W^V_h applied to sum_t p_t c_t, so
 * paged_latent_attention reads the cache's rows alone, once for all heads:
 * one cache row is the key of every head and its first latent_dim entries the
 * value.  The products with W^K and W^V are the caller's matrix products.
 *
 * Cache layout: fp16 [num_blocks][block_size][latent_dim + rope_dim],
 * contiguous: token t of sequence b is row t % block_size of block
 * block_tables[b][t / block_size]; c_t first, then r_t.  Block tables, slots,
 * ownership, errors and the error word are those of pagedkv.h.  The block
 * manager's copy-on-write works on such a cache through paged_kv_copy_blocks
 * with the cache as k_cache and as v_cache, n_kv_heads 1 and head_dim
 * latent_dim + rope_dim (both copies then carry the same bytes).
 */
#ifndef PAGEDKV_LATENT_H
#define PAGEDKV_LATENT_H

#include <stddef.h>
#include <stdint.h>

#include "pagedkv.h"
#include "pagedkv_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Norm, rotation and append of num_tokens new tokens, one kernel: for token i
 * the RMS norm (formula of pagedkv_rope.h, weight [latent_dim], NULL: none) of
 * the first latent_dim entries of its row of kv and the rotation of the last
 * rope_dim go to its cache slot; with q_rope, the position part of its queries
 * is rotated into q_out.  fp32 arithmetic, rounded once to fp16.
 *
 *  kv             device fp16, token i's latent_dim + rope_dim entries at
 *                 element i * kv_stride (the down projection's output)
 *  kv_stride      a multiple of 8, at least latent_dim + rope_dim
 *  cos_sin        device fp32 [max_positions][rope_dim], positions device
 *                 int32 [num_tokens], interleaved: as for
 *                 paged_qk_norm_rope_append with rot_dim = rope_dim
 *  q_rope, q_out  device fp16, may both be NULL (no queries): entry (i, h) of
 *                 rope_dim values at element i * token_stride + h *
 *                 head_stride; q_out may be q_rope with the same strides, and
 *                 is otherwise disjoint from it.  Strides: multiples of 8,
 *                 head strides at least rope_dim, token strides at least
 *                 (n_q_heads - 1) * head_stride + rope_dim.
 *  latent_dim     a multiple of 8, at most 1024; rope_dim a multiple of 16, at
 *                 most 256
 * Padding tokens (negative slots), bad slots and positions: as for
 * paged_qk_norm_rope_append, the token's queries included.  Pointers 16-byte
 * aligned.
 */
int paged_latent_append(const void *kv, int64_t kv_stride, const void *weight, float eps,
                        const float *cos_sin, const int32_t *positions, int max_positions,
                        int interleaved, const int64_t *slot_mapping, void *cache,
                        const void *q_rope, int64_t q_token_stride, int64_t q_head_stride,
                        void *q_out, int64_t out_token_stride, int64_t out_head_stride,
                        int n_q_heads, int num_tokens, int latent_dim, int rope_dim,
                        int block_size, int64_t num_blocks, int32_t *err_word,
                        void *cuda_stream);

/*
 * Absorbed latent attention of each sequence's newest tokens over the paged
 * cache:
 *
 *   out[i][h][:] = sum_t softmax_t(scale * q[i][h] . row_t) row_t[0:latent_dim]
 *
 * over the rows t of the token's sequence up to and including its own
 * position (the scaled logits within fp32's range).  One kernel over an even split of the batch's (sequence, query
 * rows, tokens) work, then one that joins the pieces by log-sum-exp.
 *
 *  q              device fp16 [total_q][n_q_heads][latent_dim + rope_dim]
 *  out            device fp16 [total_q][n_q_heads][latent_dim]
 *  lse_out        device fp32 [total_q][n_q_heads], natural log, may be NULL
 *  query_start    device int32 [num_seqs + 1] as for
 *                 paged_decode_attention_multi (several tokens a sequence,
 *                 causal); NULL: one token a sequence (total_q == num_seqs,
 *                 max_q_len 1), where a context length of 0 gives out = 0 and
 *                 lse = -inf
 *  max_q_len      host upper bound of the tokens of one sequence; with 0, as with
 *                 total_q 0, the call does nothing and flags nothing
 *  latent_dim     256 or 512;  rope_dim 64;  block_size 16, 32, 64, 128 or 256
 *  max_context_len, block_tables, context_lens, err_word, cuda_stream: as for
 *                 paged_decode_attention_multi
 *  workspace      device scratch of at least paged_latent_plan's bytes,
 *                 256-byte aligned; needs no zero-fill; calls that overlap in
 *                 time need separate workspaces
 * Logits, softmax and sums in fp32; the softmax weights are rounded to fp16
 * for the product with the values.  Rows behind a sequence's length are never
 * read into a result, whatever they hold; a cached row that is not finite
 * may reach every query of its sequence whose attended rows end in the same
 * 64-token tile or behind it, those before it included (their weight for it is
 * 0, and 0 times infinity is NaN).
 * A sequence whose tokens, length or rows are out of bounds sets
 * PKV_ERRBIT_CONTEXT and its rows are left unwritten; a bad block id sets
 * PKV_ERRBIT_BLOCK_ID, and the results of the sequence that names it are
 * unspecified.  At most 4096 sequences and fewer than 2^31 cache rows
 * (PKV_ERR_UNSUPPORTED beyond).  After PKV_ERRBIT_TIMEOUT every result of the call is
 * unspecified; the workspace needs nothing before the next one.
 */
int paged_latent_plan(int num_seqs, int total_q, int max_q_len, int n_q_heads, int latent_dim,
                      int rope_dim, int block_size, int max_blocks_per_seq, int max_context_len,
                      size_t *workspace_bytes_out);
int paged_latent_attention(void *out, const void *q, const void *cache,
                           const int32_t *block_tables, const int32_t *context_lens,
                           const int32_t *query_start, int num_seqs, int total_q, int max_q_len,
                           int max_blocks_per_seq, int64_t num_blocks, float scale, int n_q_heads,
                           int latent_dim, int rope_dim, int block_size, int max_context_len,
                           void *workspace, size_t workspace_bytes, float *lse_out,
                           int32_t *err_word, void *cuda_stream);

/*
 * Cached rows out of their blocks, in token order (the input of the matrix
 * product that expands them): row start[b] + j of latents and ropes, for j <
 * start[b + 1] - start[b], is row t = j of sequence b's cached tokens.
 *
 *  start          device int32 [num_seqs + 1], non-decreasing, start[0] >= 0
 *  total          rows of the outputs; rows outside [start[0],
 *                 start[num_seqs]) are left as they were
 *  latents, ropes device fp16 [total][latent_dim] and [total][rope_dim]
 *  latent_dim, rope_dim   multiples of 8, their sum at most 2048
 * A bad block id sets PKV_ERRBIT_BLOCK_ID, a token beyond max_blocks_per_seq *
 * block_size PKV_ERRBIT_CONTEXT; those rows are left as they were.
 */
int paged_latent_gather(void *latents, void *ropes, const void *cache,
                        const int32_t *block_tables, const int32_t *start, int num_seqs,
                        int64_t total, int max_blocks_per_seq, int64_t num_blocks,
                        int latent_dim, int rope_dim, int block_size, int32_t *err_word,
                        void *cuda_stream);

/*
 * Expanded latent attention of prompts (whole, or chunks behind cached
 * context), causal:
 *
 *   out[i][h] = sum_t softmax_t(scale * (q[i][h][0:d] . k[t][h] +
 *                                        q[i][h][d:] . k_rope[t])) v[t][h]
 *
 *  q              device fp16 [total_q][n_heads][head_dim + rope_dim]
 *  kv             device fp16 [total_kv][n_heads][2 * head_dim]: the head's
 *                 key k, then its value v (the product of the latents with
 *                 the expansion's weights)
 *  k_rope         device fp16 [total_kv][rope_dim], shared by all heads; with
 *                 total_kv 0, kv and k_rope may be NULL
 *  q_start, kv_start   device int32 [num_seqs + 1]: sequence b owns the query
 *                 rows [q_start[b], q_start[b + 1]), n_b of them, and the
 *                 key/value rows [kv_start[b], kv_start[b + 1]), m_b of them;
 *                 its query i sits at position m_b - n_b + i and attends the
 *                 keys up to that position.  n_b > m_b or rows out of bounds
 *                 set PKV_ERRBIT_CONTEXT, and the sequence's rows are left
 *                 unwritten.
 *  max_q_len, max_kv_len   host upper bounds of n_b and m_b (a longer sequence
 *                 is flagged as out of bounds; with max_q_len 0, as with total_q
 *                 0, the call does nothing and flags nothing).  A sequence of
 *                 more than 2^27 keys may run out a wait (PKV_ERRBIT_TIMEOUT).
 *  out            device fp16 [total_q][n_heads][head_dim];  lse_out fp32
 *                 [total_q][n_heads], may be NULL
 *  head_dim       64 or 128;  rope_dim 64
 * Needs no workspace.  Rounding as for paged_latent_attention, and so with keys
 * and values that are not finite: rows of other sequences never reach a result,
 * those of the same sequence may within a tile of 128 queries.  After
 * PKV_ERRBIT_TIMEOUT every result of the call is unspecified.
 */
int latent_prefill_attention(void *out, const void *q, const void *kv, const void *k_rope,
                             const int32_t *q_start, const int32_t *kv_start, int num_seqs,
                             int total_q, int total_kv, int max_q_len, int max_kv_len,
                             float scale, int n_heads, int head_dim, int rope_dim,
                             float *lse_out, int32_t *err_word, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_LATENT_H */
