/*
 * pagedkv_q8.h -- paged caches held in 8 bits with one scale for each block of
 * tokens and KV head.  Part of libpagedkv.so.
 *
 * Source: "Roadmap: vLLM-style serving features for TornadoVM batched decode",
 * KV-cache list ("Quantized (Q8/FP8) KV cache").  The E4M3 caches of pagedkv.h
 * have one scale for a whole tensor, which the caller has to know beforehand;
 * here the append finds the scales.
 *
 *   value of K at (block, head, row, i) = code * k_scales[block][head]
 *
 * and so for V.  Codes are E4M3 ("e4m3fn", largest 448) or int8 (-127 to 127).
 *
 * Layout: codes [num_blocks][n_kv_heads][block_size][head_dim], one byte each,
 * as in pagedkv.h; k_scales and v_scales fp32 [num_blocks][n_kv_heads].  Block
 * tables, ownership, errors and the error word are those of pagedkv.h.  Scales
 * are 0 or between 2^-100 and 2^64 (the append writes 2^-33 to 2^11 from fp16
 * where it finds none).
 *
 * Limits of every call: head_dim 64 or 128, block_size 16, 32, 64, 128 or 256,
 * at most 2048 sequences, fewer than 2^31 rows of all blocks and heads in a
 * cache, for attention about 2^31 tiles of 16 tokens and KV head by
 * max_context_len (PKV_ERR_UNSUPPORTED beyond).
 */
#ifndef PAGEDKV_Q8_H
#define PAGEDKV_Q8_H

#include <stddef.h>
#include <stdint.h>

#include "pagedkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The codes of a cache (the argument `kind`). */
#define PKV_Q8_E4M3 0
#define PKV_Q8_INT8 1

/*
 * Quantises each sequence's newest tokens as they are written to their
 * positions.  Sequence b has n_b new tokens, the last n_b of its
 * context_lens[b]; they are the rows [query_start[b], query_start[b + 1]) of
 * k_new and v_new.  For each block that they touch, each KV head, and K and V
 * apart, with limit = 448 or 127:
 *
 *   a     largest |x| of the call's new tokens in the block that is finite
 *   s0    the stored scale, where the block holds earlier tokens of the
 *         sequence (those before the new ones); 0 where it does not
 *   s     s0 = 0:  a / limit
 *         s0 > 0:  s0 * 2^k, k >= 0 the smallest with a <= s * limit
 *   codes of the new tokens: x / s to nearest even, saturated (infinities too);
 *         a NaN becomes the NaN code (E4M3) or 0 (int8).  s = 0 divides by 1
 *   k > 0: codes of the earlier tokens become code * 2^-k to nearest even
 *
 * (a / limit, a / (s0 * limit) and x / s each rounded once to fp32.)  Growth by
 * powers of two leaves E4M3 codes exact but for subnormal results, and int8
 * ones off by at most one step of the final scale, however many tokens came one
 * by one.  Rows of a block behind the new tokens are left as they were.
 *
 *  k_new, v_new   device fp16, token i's n_kv_heads * head_dim entries at
 *                 element i * stride (columns of a fused projection's output)
 *  k_stride, v_stride   multiples of 8, at least n_kv_heads * head_dim
 *  query_start    device int32 [num_seqs + 1], non-decreasing, or NULL: one
 *                 token a sequence (total == num_seqs, max_q_len 1), where a
 *                 context length of 0 is a sequence without a token
 *  total          rows of k_new and v_new
 *  max_q_len      host upper bound of n_b; with 0, as with total 0, the call
 *                 does nothing and flags nothing
 * A sequence with n_b outside [0, max_q_len], n_b > context_lens[b], rows
 * outside [0, total) or a length beyond max_blocks_per_seq * block_size sets
 * PKV_ERRBIT_CONTEXT and nothing of it is written (the others are, also where
 * starts decrease); a bad block id sets PKV_ERRBIT_BLOCK_ID and that block is
 * left out.  Two sequences that write to one block in one call race
 * (copy-on-write first: paged_kv_copy_blocks_q8).
 * Pointers 16-byte aligned (tables and lengths: 4).
 */
int paged_kv_append_q8(const void *k_new, const void *v_new, int64_t k_stride, int64_t v_stride,
                       const int32_t *query_start, const int32_t *block_tables,
                       const int32_t *context_lens, int num_seqs, int total, int max_q_len,
                       int max_blocks_per_seq, void *k_cache, void *v_cache, float *k_scales,
                       float *v_scales, int kind, int n_kv_heads, int head_dim, int block_size,
                       int64_t num_blocks, int32_t *err_word, void *cuda_stream);

/*
 * Attention of each sequence's newest tokens over the codes:
 *
 *   out[i][h] = sum_t softmax_t(scale * q[i][h] . k_t) v_t
 *
 * over the tokens t of the sequence up to and including the query's own
 * position; query head h reads KV head h / (n_q_heads / n_kv_heads), any
 * whole ratio up to 128 (PKV_ERR_UNSUPPORTED beyond).  Up to 32 query rows of
 * a KV head (max_q_len times that ratio) are streamed through one kernel; more
 * go in tiles of 128 rows to another, on tcgen05 (max_context_len, or with 0
 * the tables' tokens, up to 2^25 there, PKV_ERR_UNSUPPORTED beyond).  max_q_len
 * decides for the whole call: a decode batch with a chunk in it is better given
 * in two calls (64 sequences of one new token and one of 512: 125 us in one, 75
 * in two; next to a chunk each of those costs a tile of 128 rows).  out and q
 * do not overlap.
 *
 *  q              device fp16, token i's n_q_heads * head_dim entries at
 *                 element i * q_stride (a multiple of 8)
 *  out            device fp16 [total_q][n_q_heads][head_dim]
 *  lse_out        device fp32 [total_q][n_q_heads], natural log, may be NULL
 *  query_start    device int32 [num_seqs + 1] as for
 *                 paged_decode_attention_multi (n_b new tokens, causal), or
 *                 NULL: one token a sequence (total_q == num_seqs, max_q_len
 *                 1), where a context length of 0 gives out = 0, lse = -inf
 *  max_q_len      host upper bound of n_b; with 0, as with total_q 0, the call
 *                 does nothing and flags nothing
 *  max_context_len, block_tables, context_lens, err_word, cuda_stream: as for
 *                 paged_decode_attention_multi
 *  workspace      device scratch of at least paged_decode_q8_plan's bytes,
 *                 256-byte aligned.  A plan's bytes are enough for every call
 *                 with the same n_kv_heads and head_dim whose other sizes are
 *                 no larger: one for a loop's largest call serves the loop.
 *                 Its first PKV_WORKSPACE_COUNTER_BYTES bytes hold arrival
 *                 counters: zero before the first use, and left at zero by
 *                 every call, also by one that flags PKV_ERRBIT_TIMEOUT.  After
 *                 PKV_ERRBIT_WORKSPACE (a counter that did not start at zero)
 *                 clear them with paged_decode_workspace_clear.  Calls that
 *                 overlap in time need separate workspaces.
 *  flags          0 or PKV_TABLES_READY, which covers query_start too, and
 *                 err_word where the kernel before clears it (made use of up
 *                 to 32 rows)
 * Logits, softmax and sums in fp32; the weights times their block's V scale
 * are rounded to fp16 for the product with the codes, which are exact: off by
 * 2^-11 of themselves, or where that is more by 2^-19 of the block's V scale
 * (with more than 32 rows: of the largest V scale among 64 tokens; of 2^-26 at
 * least), the largest weight of the row being 1.  Rows
 * behind a sequence's length never reach a result, whatever they hold.  A
 * cached NaN makes the queries that attend it NaN; one of a sequence's newest
 * tokens may also reach that sequence's earlier queries.
 * A sequence whose tokens, length or rows are out of bounds sets
 * PKV_ERRBIT_CONTEXT and its rows are left unwritten; a bad block id sets
 * PKV_ERRBIT_BLOCK_ID, and that sequence's results are unspecified.
 */
int paged_decode_q8_plan(int num_seqs, int total_q, int max_q_len, int n_q_heads, int n_kv_heads,
                         int head_dim, int block_size, int max_blocks_per_seq,
                         int max_context_len, size_t *workspace_bytes_out);
int paged_decode_attention_q8(void *out, const void *q, int64_t q_stride, const void *k_cache,
                              const void *v_cache, const float *k_scales, const float *v_scales,
                              int kind, const int32_t *block_tables, const int32_t *context_lens,
                              const int32_t *query_start, int num_seqs, int total_q,
                              int max_q_len, int max_blocks_per_seq, int64_t num_blocks,
                              float scale, int n_q_heads, int n_kv_heads, int head_dim,
                              int block_size, int max_context_len, void *workspace,
                              size_t workspace_bytes, float *lse_out, int32_t *err_word,
                              void *cuda_stream, uint32_t flags);

/*
 * Cached tokens back in fp16, in token order: row start[b] + j of k and v is
 * token j of sequence b, j < start[b + 1] - start[b], value = code * scale
 * rounded to fp32 and that to fp16, each to nearest even, at most 65504 in size
 * (one product in some 20000 has more bits than fp32 and lands next to a tie of
 * fp16: there the two roundings differ from one).
 *  start          device int32 [num_seqs + 1], non-decreasing, start[0] >= 0
 *                 (rows that two sequences have in common are unspecified)
 *  total          rows of the outputs; rows outside [start[0],
 *                 start[num_seqs]) are left as they were
 *  k, v           device fp16 [total][n_kv_heads][head_dim]
 * A bad block id sets PKV_ERRBIT_BLOCK_ID, a token beyond max_blocks_per_seq *
 * block_size PKV_ERRBIT_CONTEXT; those rows are left as they were.
 */
int paged_kv_gather_q8(void *k, void *v, const void *k_cache, const void *v_cache,
                       const float *k_scales, const float *v_scales, int kind,
                       const int32_t *block_tables, const int32_t *start, int num_seqs,
                       int64_t total, int max_blocks_per_seq, int64_t num_blocks,
                       int n_kv_heads, int head_dim, int block_size, int32_t *err_word,
                       void *cuda_stream);

/*
 * paged_kv_copy_blocks of such caches: codes of rows [0, tokens[i]) (all rows
 * with tokens NULL) and the scales of every KV head from block src[i] to block
 * dst[i].  Errors and races as there; tokens[i] = 0 copies the scales alone.
 */
int paged_kv_copy_blocks_q8(void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                            const int32_t *src, const int32_t *dst, const int32_t *tokens,
                            int num_copies, int n_kv_heads, int head_dim, int block_size,
                            int64_t num_blocks, int32_t *err_word, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_Q8_H */
