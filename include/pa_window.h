/*
 * pa_window.h — part of libpa's C ABI: the cache write with the position
 * rotation applied on the way, attention with a sliding window and a few
 * first tokens that stay visible, and a KV cache held in 8 bits with one
 * scale per block of tokens and head.
 *
 * What sets these entry points apart from those of pa.h:
 *   - 16-bit arrays are fp16 or bf16 (pa_dtype);
 *   - grouped heads: num_heads = G * num_kv_heads query heads, query head h
 *     reads K/V head h / G (G = 1 is pa.h's case; G <= 128);
 *   - a query at position p sees position t when
 *         t <= p  and  (t > p - window  or  t < num_sinks).
 *     window >= 1 (the query's own position counts), num_sinks >= 0; a window
 *     of max_context_len or more is the whole context.  Block-table entries
 *     of blocks that hold no position some query of the call sees are never
 *     read, so blocks that the window has left may have been given back to
 *     the pool (any entry, -1 for example).
 *
 * Layouts (row-major, device pointers, 16-byte aligned unless said otherwise):
 *   q, out            [num_tokens, num_heads, head_dim]
 *   k_cache, v_cache  [num_blocks, num_kv_heads, block_size, head_dim]
 *   k_codes, v_codes  the same shape, one byte a value (pa_kv8_type)
 *   kv_scales         [num_blocks, num_kv_heads rounded up to even, 2] float:
 *                     (s_k, s_v) of each block and head; a value is s * code.
 *                     (Rounded up so that a block's scales are a multiple of
 *                     16 bytes and pa_copy_blocks_raw / pa_swap_blocks move
 *                     them as they move the codes.)
 *   block_tables, context_lens, slot_mapping, query_start_loc as in pa.h
 * head_dim 64 or 128 and block_size 8, 16, 32, 64 or 128 (else
 * PA_ERR_UNSUPPORTED).  Ownership, streams, asynchronous execution and the
 * device error word are as in pa.h.
 */
#ifndef PA_WINDOW_H
#define PA_WINDOW_H

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_dtype {
    PA_F16 = 0,
    PA_BF16 = 1
} pa_dtype;

/* Codes of the 8-bit cache: two's complement integers in [-127, 127], or
 * e4m3 numbers (4 exponent and 3 mantissa bits, largest 448). */
typedef enum pa_kv8_type {
    PA_KV8_INT8 = 0,
    PA_KV8_E4M3 = 1
} pa_kv8_type;

/* Bit of the device error word: a position outside [0, max_position). */
#define PA_DEVERR_POSITION 32u

/*
 * Rotate each token's query and key rows by its position and write key and
 * value into the paged cache.  For token i with slot_mapping[i] >= 0 and the
 * table row (c, s) = cos_sin[positions[i]]:
 *     y[a] = x[a] c[j] - x[b] s[j],   y[b] = x[b] c[j] + x[a] s[j]
 * for every pair j < rotary_dim / 2, where (a, b) = (j, j + rotary_dim / 2),
 * or (2j, 2j + 1) when `interleaved` is not 0; the other dims are copied.
 * q's rotated rows go to q_out (which may be q itself, with the same stride),
 * key's to k_cache and value's unrotated rows to v_cache at the token's slot.
 * A token with a negative slot is padding: nothing of it is written, its q_out
 * row included.
 *   cos_sin    [max_position, rotary_dim] float: the cosines of the
 *              rotary_dim / 2 angles, then their sines
 *   positions  [num_tokens] int64
 *   *_stride   elements from one token's rows to the next one's (a multiple
 *              of 8, at least heads * head_dim), so that q, key and value may
 *              be parts of one projection's output
 * rotary_dim is a multiple of 16 in [0, head_dim] (else PA_ERR_UNSUPPORTED);
 * 0 rotates nothing and cos_sin and positions may be NULL (else max_position
 * is at least 1).  The arithmetic is
 * in fp32, each product and sum rounded by itself, then rounded once to the
 * 16-bit type.  A slot outside the pool or a position outside the table is
 * recorded (PA_DEVERR_SLOT, PA_DEVERR_POSITION) and the token skipped.  Slots
 * of one call must be distinct.  num_tokens == 0 is a no-op.
 */
PA_API pa_status pa_rope_and_cache(void *q_out, int64_t q_out_stride, const void *q,
                                   int64_t q_stride, const void *key, int64_t key_stride,
                                   const void *value, int64_t value_stride, void *k_cache,
                                   void *v_cache, const float *cos_sin, int rotary_dim,
                                   int max_position, int interleaved, const int64_t *positions,
                                   const int64_t *slot_mapping, int num_tokens, int num_heads,
                                   int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                   pa_dtype dtype, pa_stream_t stream);

/*
 * pa_rope_and_cache into the 8-bit cache.  The rotated key and the value are
 * quantized from fp32: code = round(x / s) (half to even; |code| <= 127, or
 * the nearest e4m3 number up to 448).  Blocks fill from their first row: the
 * tokens that a call brings for one block stand next to each other in the
 * batch, in consecutive slots, and the rows before them are what the block
 * already holds.  With m the largest |x| of the new rows and `top` 127 or 448:
 *     s = m / top                     when the new rows start at row 0,
 *     s = max(the block's s, m / top) otherwise; where s grows, the older
 *                                     rows become round(code * (s_old / s)).
 * (Where s is new, x / s is taken as x top / m, before s is rounded to fp32;
 * so too where s lies below the normal numbers and x / s would pass the top.)
 * Rows behind the new ones keep their codes (a later write replaces them).
 * A block whose rows are all zero has s = 0 and codes 0.  Rows holding inf or
 * NaN make their block's values unspecified.  A block is written by one run
 * of tokens per call: one that the call's tokens come back to (interleaved
 * sequences, a slot given twice) is recorded (PA_DEVERR_SLOT) and its values
 * unspecified.  Other arguments and rules as pa_rope_and_cache; a
 * position outside the table is recorded and its row's values unspecified.
 */
PA_API pa_status pa_rope_and_cache_q8(void *q_out, int64_t q_out_stride, const void *q,
                                      int64_t q_stride, const void *key, int64_t key_stride,
                                      const void *value, int64_t value_stride, void *k_codes,
                                      void *v_codes, float *kv_scales, const float *cos_sin,
                                      int rotary_dim, int max_position, int interleaved,
                                      const int64_t *positions, const int64_t *slot_mapping,
                                      int num_tokens, int num_heads, int num_kv_heads,
                                      int head_dim, int block_size, int num_blocks,
                                      pa_dtype dtype, pa_kv8_type kv_type, pa_stream_t stream);

/*
 * Bytes of workspace pa_decode_window and pa_decode_q8 need: partial results
 * of the contexts that are split between blocks of threads (34 MB), and one
 * merge counter per (sequence, K/V head, 8 or 16 query heads); the same for
 * every head_dim.  Never 0.  Zero it once before its first use
 * (pa_decode_workspace_init); every completed call leaves it ready for the
 * next, of any size that fits it (after PA_DEVERR_TIMEOUT, zero it again).
 * Calls that share a workspace must not overlap on the GPU (this holds for
 * replayed graphs too).
 */
PA_API size_t pa_decode_window_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                              int head_dim);

/*
 * One query per sequence (the newest token, p = context_lens[b] - 1) over a
 * 16-bit cache:
 *     out[b, h, :] = sum_t exp(s_t - max s) V_t / sum_t exp(s_t - max s),
 *     s_t = scale * sum_d q[b, h, d] * K_t[d],  over the positions t it sees.
 * Scores, softmax statistics and sums are fp32; the weights enter the product
 * with V as the sum of two numbers of the cache's 16-bit type (within 2^-15 of
 * fp32's value), or as one where query heads are taken 16 at a time (groups of
 * more than 8, and more than 32 units of sequence, K/V head and 16 of its query
 * heads).  L == 0 writes zeros.  What positions
 * that are not seen hold has no effect.  max_context_len bounds
 * context_lens and must not exceed max_blocks_per_seq * block_size or 2^30.  Results
 * do not depend on the order in which blocks of threads run.
 */
PA_API pa_status pa_decode_window(void *out, const void *q, const void *k_cache,
                                  const void *v_cache, const int32_t *block_tables,
                                  int max_blocks_per_seq, const int32_t *context_lens,
                                  int max_context_len, int window, int num_sinks, int num_seqs,
                                  int num_heads, int num_kv_heads, int head_dim, int block_size,
                                  int num_blocks, pa_dtype dtype, float scale, void *workspace,
                                  size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_decode_window over the 8-bit cache: K_t = s_k * code, V_t = s_v * code
 * with the scales of the block and head that hold t; q and out in `dtype`.  The
 * weights enter the product with V times s_v, in fp16 numbers (as many as
 * there) relative to the largest: what is below 2^-31 of it is lost.
 * About half the bytes of pa_decode_window.
 */
PA_API pa_status pa_decode_q8(void *out, const void *q, const void *k_codes, const void *v_codes,
                              const float *kv_scales, const int32_t *block_tables,
                              int max_blocks_per_seq, const int32_t *context_lens,
                              int max_context_len, int window, int num_sinks, int num_seqs,
                              int num_heads, int num_kv_heads, int head_dim, int block_size,
                              int num_blocks, pa_dtype dtype, pa_kv8_type kv_type, float scale,
                              void *workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * The same attention for several queries a sequence (prompts, chunks that
 * continue a cached context, draft tokens): the last n_b =
 * query_start_loc[b+1] - query_start_loc[b] of sequence b's context_lens[b]
 * cached tokens are its queries, at positions L - n_b + i, as in pa_prefill.
 * Runs on the tensor cores (tcgen05); scores and sums fp32, the weights enter
 * the product with V in the cache's 16-bit type.  scale must be finite and
 * > 0.  Rows of q and out that belong to no sequence are left as they are.
 * A V row that is not finite, and that some query of its sequence sees, may
 * also reach queries less than 256 positions away from such a query, though
 * the mask hides it from them (a weight of zero times infinity is NaN); rows
 * that no query sees have no effect.  n_b < 0, > L_b or > max_query_len,
 * or rows outside q, are recorded (PA_DEVERR_CONTEXT_LEN) and that sequence
 * is skipped.
 */
PA_API pa_status pa_prefill_window(void *out, const void *q, const void *k_cache,
                                   const void *v_cache, const int32_t *block_tables,
                                   int max_blocks_per_seq, const int32_t *context_lens,
                                   int max_context_len, const int32_t *query_start_loc,
                                   int num_tokens, int max_query_len, int window, int num_sinks,
                                   int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                   int block_size, int num_blocks, pa_dtype dtype, float scale,
                                   pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_WINDOW_H */
