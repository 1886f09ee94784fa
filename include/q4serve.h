/*
 * q4serve.h -- C ABI of the operators around the 4-bit linear layer in a
 * decoder: the paged 8-bit key/value cache, attention over it, and token log
 * probabilities of the output head's logits with their gradient.  They are
 * part of the same library as q4linear.h and share its status codes and its
 * conventions: device pointers owned by the caller, nothing allocated or
 * kept, work queued on `stream`, every host-visible argument checked before
 * anything is queued, deterministic results.
 *
 * The cache of one layer
 *   k_cache  int8  [pages, kv_heads, page, head_dim]
 *   v_cache  int8  [pages, kv_heads, head_dim, page]  (tokens innermost: the
 *                  attention kernel feeds 16 tokens of one value column
 *                  straight into a matrix operand)
 *   k_scale, v_scale  float [pages, kv_heads]
 * all contiguous, caches 16-byte aligned.  A scale covers one page of one
 * head: an element stands for code * scale, codes in [-127, 127], scale >= 0
 * (a negative scale is none: its page's values are NaN in every function).
 * page is 16, 32, 64 or 128 tokens; head_dim a multiple of 16 up to 256.
 *
 * Sequences are ragged and packed.  Sequence b (0 <= b < batch) owns the new
 * tokens cu_new[b] .. cu_new[b + 1] - 1 of this call (cu_new[0] = 0,
 * cu_new[batch] = T, not decreasing) and has lengths[b] tokens in all, the
 * new ones last: new token i of sequence b is at position
 *   pos = lengths[b] - (cu_new[b + 1] - cu_new[b]) + i.
 * Position p lies in slot p % page of page page_table[b * table_ld +
 * p / page].  cu_new, lengths and page_table are device int32 arrays, so a
 * captured graph can be replayed with new values in them.
 *
 * What the host cannot see is checked in the kernels, which never read or
 * write outside the arrays: see each function for what a page number outside
 * [0, pages) or a position past max_pages does.
 */
#ifndef Q4SERVE_H
#define Q4SERVE_H

#include "q4linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of these operators: Q4_DTYPE_F32, Q4_DTYPE_F16 and */
#define Q4_DTYPE_BF16 2

/*
 * q4_kv_append -- new keys and values into the cache, the keys (and, if
 * given, the queries) turned by their position on the way.
 *
 *   k, v    [T, kv_heads, head_dim] of `dtype`; token stride *_ts and head
 *           stride *_hs in elements, head_dim contiguous
 *   q       [T, heads, head_dim] or NULL; q_out likewise, may be q itself
 *           (the same pointer and strides), else must not overlap an input.
 *           In place, the queries may lie in one array with k and v (rows of
 *           a fused projection, heads of either interleaved with the others'),
 *           of the same token stride and without an element in common
 *   inv_freq  float [rot / 2], or NULL with rot == 0 (no rotation)
 *   rot     even, 0 <= rot <= head_dim: elements of a head that turn.  Pair
 *           i is elements (i, i + rot / 2), or (2 i, 2 i + 1) if
 *           interleaved, and (a, b) becomes (a c - b s, a s + b c) with the
 *           cosine and sine of pos * inv_freq[i].  The angle is formed and
 *           reduced in 64 bits, so far positions keep their precision; the
 *           products are fp32.
 *   max_new   upper bound of the new tokens of one sequence (T always is
 *           one); it sizes the launch.  Of a sequence with more, the first
 *           max_new are stored (queries are turned all the same).
 *
 * For each page and head that gets new tokens, with s the scale it had (0
 * if slot 0 is among the new ones: the page starts anew) and A the largest
 * magnitude among its new elements:
 *   s' = max(s, A / 127);  codes it held -> rint(code * (s / s'));
 *   new codes = clamp(rint(x / s'), -127, 127);  all 0 if s' == 0.
 * The other slots of a page that starts anew become 0.  A NaN or infinity
 * among the new elements makes s' NaN or infinite, so that the page's values
 * are not finite until the page starts anew.
 * A token whose page number is outside [0, pages), whose position is
 * negative or past max_pages * page, is not stored.  No two sequences may
 * append to the same page in one call.
 *
 * T == 0 or batch == 0 is a no-op.
 */
q4_status q4_kv_append(const void *k, int64_t k_ts, int64_t k_hs,
                       const void *v, int64_t v_ts, int64_t v_hs,
                       const void *q, int64_t q_ts, int64_t q_hs,
                       void *q_out, int64_t qo_ts, int64_t qo_hs,
                       int32_t dtype, int64_t T, int64_t batch,
                       int64_t heads, int64_t kv_heads, int64_t head_dim,
                       int8_t *k_cache, int8_t *v_cache, float *k_scale,
                       float *v_scale, int64_t pages, int64_t page,
                       const int32_t *page_table, int64_t table_ld,
                       int64_t max_pages, const int32_t *cu_new,
                       const int32_t *lengths, int64_t max_new,
                       const float *inv_freq, int64_t rot,
                       int32_t interleaved, void *stream);

/*
 * q4_kv_dequant -- the values of a whole cache, code * scale rounded once to
 * `dtype`: k, v [pages, kv_heads, page, head_dim], contiguous and 16-byte
 * aligned (the values in token order too).
 */
q4_status q4_kv_dequant(const int8_t *k_cache, const int8_t *v_cache,
                        const float *k_scale, const float *v_scale,
                        int64_t pages, int64_t kv_heads, int64_t page,
                        int64_t head_dim, int32_t dtype, void *k, void *v,
                        void *stream);

/*
 * q4_attention -- attention of the new tokens over their sequence's cache
 * (the new tokens themselves included: append first):
 *
 *   out[t, h] = sum_j p_j v_j,  p = softmax_j(scale * q[t, h] . k_j)
 *
 * over the positions j <= pos(t), and j > pos(t) - window if window > 0, of
 * kv head h / (heads / kv_heads).  A query that sees no position (a length
 * of 0) gives 0.
 *
 *   q, out  [T, heads, head_dim] of `dtype` with token and head strides;
 *           out must not overlap an input
 *   max_new   upper bound of the new tokens of one sequence: queries past
 *           it are not computed, their outputs left as they are.  With
 *           batch it sizes the launch: of more than 2^24 - 1 workgroups the
 *           call is refused (about 8000 sequences with max_new = T)
 *   max_len   upper bound of lengths: it sizes the launch and the
 *           workspace.  Positions past it are not attended.
 *   workspace   q4_attention_workspace_bytes(...) bytes, 16-byte aligned
 *           (may be NULL when that is 0)
 *
 * Positions at or past lengths[b] and outside the window are never read, so
 * their slots, pages and table entries may hold anything.  A visible
 * position whose page number is outside [0, pages) or whose position is past
 * max_pages * page makes the outputs that see it NaN.  So does a page's key
 * scale that is not finite; outputs that see a value scale that is not finite
 * are not finite.
 *
 * Arithmetic: integer dot products of the 8-bit codes with q and p held as
 * fixed-point numbers of four 8-bit digits (fp32 queries; three digits for
 * 16-bit ones) below the largest of the query's row and of the tile, summed
 * exactly in int32 over each tile of 64 tokens; scales, softmax statistics and
 * sums over tiles in fp32.
 */
q4_status q4_attention(const void *q, int64_t q_ts, int64_t q_hs, void *out,
                       int64_t o_ts, int64_t o_hs, int32_t dtype, int64_t T,
                       int64_t batch, int64_t heads, int64_t kv_heads,
                       int64_t head_dim, const int8_t *k_cache,
                       const int8_t *v_cache, const float *k_scale,
                       const float *v_scale, int64_t pages, int64_t page,
                       const int32_t *page_table, int64_t table_ld,
                       int64_t max_pages, const int32_t *cu_new,
                       const int32_t *lengths, int64_t max_new,
                       int64_t max_len, float scale, int64_t window,
                       void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace q4_attention needs (0 if none, or invalid sizes). */
size_t q4_attention_workspace_bytes(int32_t dtype, int64_t T, int64_t batch,
                                    int64_t heads, int64_t kv_heads,
                                    int64_t head_dim, int64_t page,
                                    int64_t max_new, int64_t max_len,
                                    int64_t window);

/*
 * q4_token_logprobs -- for each row of logits [M, vocab] (row pitch ld, in
 * elements of `dtype`):
 *   lse      = log sum_v exp(x_v)
 *   logprob  = x[target] - lse
 *   entropy  = -sum_v p_v log p_v,  p_v = exp(x_v - lse)
 *   top_ids, top_logprobs [M, top_k]: the top_k largest logits in descending
 *              order, equal ones by ascending index, and their x - lse
 * in fp32, sums in fp32, one pass over the logits.  vocab is at most 2^30.
 *   targets  int64 [M] or NULL (then logprob is not written).  A negative
 *            target stands for none: logprob 0.  One >= vocab gives NaN.
 *   top_k    0 .. 32, at most vocab
 * -inf is an impossible token (p = 0).  A row of nothing but -inf gives lse
 * and logprob -inf and entropy 0.  A NaN or +inf in a row makes its lse,
 * logprob, entropy and top_logprobs NaN; NaNs are not alternatives (missing
 * ones have index -1).
 */
q4_status q4_token_logprobs(const void *logits, int64_t ld, int32_t dtype,
                            int64_t M, int64_t vocab, const int64_t *targets,
                            int64_t top_k, float *logprob, float *entropy,
                            float *lse, int64_t *top_ids,
                            float *top_logprobs, void *workspace,
                            size_t workspace_bytes, void *stream);

/* Bytes of workspace q4_token_logprobs needs (0 if none, or invalid sizes). */
size_t q4_token_logprobs_workspace_bytes(int64_t M, int64_t vocab,
                                         int64_t top_k, int32_t dtype);

/*
 * q4_token_logprobs_backward -- the gradient of logprob and entropy:
 *   dlogits[m, v] = g_logprob[m] (1[v == target] - p_v)
 *                   - g_entropy[m] p_v (log p_v + entropy[m])
 * with p_v = exp(x_v - lse[m]); lse and entropy as q4_token_logprobs gave
 * them.  dlogits is of the logits' type and may be the logits themselves
 * (same pointer and pitch), else must not overlap an input.
 *   g_logprob, g_entropy  float [M]; either may be NULL (0), not both
 * A row with a negative target has no g_logprob term, one with a target
 * >= vocab becomes NaN, one of nothing but -inf becomes 0.
 */
q4_status q4_token_logprobs_backward(const void *logits, int64_t ld,
                                     int32_t dtype, int64_t M, int64_t vocab,
                                     const int64_t *targets, const float *lse,
                                     const float *entropy,
                                     const float *g_logprob,
                                     const float *g_entropy, void *dlogits,
                                     int64_t ldd, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4SERVE_H */
