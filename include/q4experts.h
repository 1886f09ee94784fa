/*
 * q4experts.h -- C ABI of the operators around packed experts and the packed
 * output head: routing tokens to experts, the experts' gated feed-forward over
 * 4-bit weights, and the head's softmax cross entropy without its logits,
 * each with its gradient.  They are part of the same library as q4linear.h
 * and share its status codes and its conventions: device pointers owned by
 * the caller, nothing allocated or kept, work queued on `stream`, every
 * host-visible argument checked before anything is queued, deterministic
 * results.
 *
 * Packed weights are those of q4_linear, contiguous, one matrix after the
 * other for experts: codes uint8 [E, N, K / 2] (4-byte aligned) and scales
 * float [E, ceil(K / group_size), N], or [E, N] when group_size is 0 (a scale
 * per row).  K (hidden, width) is a multiple of 8 up to 32768; group_size is
 * 0, 32 or a multiple of 64 (others: Q4_ERR_UNSUPPORTED).  A group_size >= K is
 * one group.  Weights are constants: gradients are those of the activations.
 *
 * Arithmetic: binary16 operands on MFMA with fp32 sums.  A weight's code is
 * exact in binary16.  A row of activations is scaled by a power of two to the
 * top of binary16's range, so that no magnitude overflows, and held as one
 * binary16 number (16-bit types: bf16 and fp16 values are exact) or as two
 * (fp32, and for every type what is computed on the way: 22 bits), no finer
 * than 2^-39 of its row's largest.  Forward, a scale multiplies fp32 sums.
 * Backward, a row's gradient times the scale (formed in fp32) is held as two, no
 * finer than 2^-39 of its row's largest (for the head |g_loss|) times the
 * largest scale of its group.
 * Infinities and NaN of a row reach no other row; an infinite element makes
 * its row's results infinite or NaN.  A workspace may serve any number of
 * calls one after the other, from captured graphs too, but no two at once.
 */
#ifndef Q4EXPERTS_H
#define Q4EXPERTS_H

#include "q4linear.h"
#include "q4serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scores of q4_route. */
#define Q4_SCORE_SOFTMAX 0
#define Q4_SCORE_SIGMOID 1

/*
 * q4_route -- the experts of each token and their weights.
 *
 *   logits   [T, experts] of `dtype`, row pitch ld in elements
 *   bias     float [experts] or NULL: added to the scores for the choice
 *            alone (the weights are the scores')
 *   groups   divides experts; expert e is in group e / (experts / groups)
 *
 * With s = softmax or sigmoid of the logits, an expert's value is s (without
 * a bias: its logit, which has the same order) or s + bias, formed in 64 bits
 * so that rounding decides no choice.  An expert whose logit or value is -inf
 * is not eligible; NaN ranks below every number.  With groups > 1 the
 * top_groups groups of the largest group value stay: the value of a group's best
 * expert, with a bias the sum of its two best.  Of the experts left, the top_k of the
 * largest values are chosen, in descending order; ties, also between groups,
 * go to the lowest index.
 *   ids      int32 [T, top_k]; -1 where fewer are eligible
 *   weights  float [T, top_k]: scale * s, divided by the sum of the chosen s
 *            if renormalize (however small they are); 0 where the id is -1
 * A NaN in a row, or a +inf under softmax, makes the row's weights NaN.
 * T < 2^24, experts <= 1024, top_k <= 32, top_k <= experts / groups *
 * top_groups.
 */
q4_status q4_route(const void *logits, int64_t ld, int32_t dtype, int64_t T,
                   int64_t experts, int64_t top_k, int32_t score,
                   const float *bias, int64_t groups, int64_t top_groups,
                   int32_t renormalize, float scale, int32_t *ids,
                   float *weights, void *stream);

/*
 * q4_route_backward -- the gradient of sum(g_weights * weights) with respect
 * to the logits, the choice held fixed.
 *   ids        as q4_route gave them (a negative one stands for none; one >=
 *              experts makes the row's gradient NaN)
 *   g_weights  float [T, top_k]
 *   dlogits    [T, experts] of the logits' type; may be the logits themselves
 *              (same pointer and pitch), else must not overlap an input
 */
q4_status q4_route_backward(const void *logits, int64_t ld, int32_t dtype,
                            int64_t T, int64_t experts, int64_t top_k,
                            const int32_t *ids, int32_t score,
                            int32_t renormalize, float scale,
                            const float *g_weights, void *dlogits,
                            int64_t ldd, void *stream);

/*
 * q4_experts -- the gated feed-forward of each token's experts:
 *
 *   out[t] = sum_j weights[t, j] * down_e (silu(gate_e x[t]) * (up_e x[t])),
 *            e = ids[t, j]
 *
 *   x        [T, hidden] of `dtype`, row pitch ldx
 *   ids      int32 [T, top_k]; a negative one is an empty slot, one >=
 *            experts makes its token's output NaN.  The same expert may
 *            stand in several slots
 *   gate_up  packed [experts, 2 * width, hidden / 2]: rows 0 .. width - 1 are
 *            the gate's, the rest up's
 *   down     packed [experts, hidden, width / 2]
 *   out      [T, hidden] of `dtype`, row pitch ldo; a token of empty slots
 *            is 0
 *   pre      float [T, top_k, 2 * width] or NULL: receives gate and up before
 *            the product, which q4_experts_backward takes (empty slots are
 *            left as they are)
 *   workspace  q4_experts_workspace_bytes(...) bytes, 16-byte aligned
 * The sum over slots is in slot order.  experts <= 1024, top_k <= 32,
 * T * top_k < 2^24; a call of more than 2^23 tiles (64 rows by 128 columns of
 * hidden or 2 * width) is refused.
 */
q4_status q4_experts(const void *x, int64_t ldx, int32_t dtype, int64_t T,
                     int64_t hidden, int64_t width, int64_t experts,
                     int64_t top_k, const int32_t *ids, const float *weights,
                     const uint8_t *gate_up, const float *gate_up_scales,
                     const uint8_t *down, const float *down_scales,
                     int64_t group_size, int32_t nibble_order, void *out,
                     int64_t ldo, float *pre, void *workspace,
                     size_t workspace_bytes, void *stream);

/* Bytes of workspace q4_experts needs (0 for invalid sizes). */
size_t q4_experts_workspace_bytes(int32_t dtype, int64_t T, int64_t hidden,
                                  int64_t width, int64_t experts,
                                  int64_t top_k, int64_t group_size);

/*
 * q4_experts_backward -- the gradients of sum(dout * out) with respect to x
 * and weights.
 *   dout      [T, hidden] of `dtype`, row pitch lddo
 *   pre       as q4_experts gave it for the same x and ids
 *   dx        [T, hidden] of `dtype`, row pitch lddx
 *   dweights  float [T, top_k]; 0 for an empty slot
 * An id >= experts makes its token's dx and its own dweights NaN.  Limits as
 * q4_experts', of tiles 2^24 - 1.
 */
q4_status q4_experts_backward(const void *dout, int64_t lddo, int32_t dtype,
                              int64_t T, int64_t hidden, int64_t width,
                              int64_t experts, int64_t top_k,
                              const int32_t *ids, const float *weights,
                              const float *pre, const uint8_t *gate_up,
                              const float *gate_up_scales,
                              const uint8_t *down, const float *down_scales,
                              int64_t group_size, int32_t nibble_order,
                              void *dx, int64_t lddx, float *dweights,
                              void *workspace, size_t workspace_bytes,
                              void *stream);

/* Bytes of workspace q4_experts_backward needs (0 for invalid sizes). */
size_t q4_experts_backward_workspace_bytes(int32_t dtype, int64_t T,
                                           int64_t hidden, int64_t width,
                                           int64_t experts, int64_t top_k,
                                           int64_t group_size);

/*
 * q4_head_cross_entropy -- for each row of x, with z = W x the packed head's
 * logits (never stored):
 *   lse  = log sum_v exp(z_v),  loss = lse - z[target]
 *
 *   x        [M, K] of `dtype`, row pitch ldx
 *   qw       packed [vocab, K / 2]; scales as above
 *   targets  int64 [M]; a negative one stands for none: loss 0 (lse is
 *            given all the same).  One >= vocab gives a NaN loss
 *   workspace  q4_head_cross_entropy_workspace_bytes(...) bytes, 16-byte
 *            aligned
 * M < 2^24, vocab <= 2^30; a call of more than 2^24 - 1 tiles (64 or 128 rows,
 * of at most 8192, by 128 columns) is refused, as by the gradient.
 */
q4_status q4_head_cross_entropy(const void *x, int64_t ldx, int32_t dtype,
                                int64_t M, int64_t vocab, int64_t K,
                                const uint8_t *qw, const float *scales,
                                int64_t group_size, int32_t nibble_order,
                                const int64_t *targets, float *loss,
                                float *lse, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Bytes of workspace q4_head_cross_entropy needs (0 for invalid sizes). */
size_t q4_head_cross_entropy_workspace_bytes(int32_t dtype, int64_t M,
                                             int64_t vocab, int64_t K,
                                             int64_t group_size);

/*
 * q4_head_cross_entropy_backward -- the gradient of sum(g_loss * loss) with
 * respect to x:
 *   dx[m, k] = g_loss[m] * sum_v (p_v - 1[v == target]) W[v, k]
 * in pieces of the vocabulary, whose logits are computed again.
 *   lse      as q4_head_cross_entropy gave it
 *   g_loss   float [M]
 *   dx       [M, K] of `dtype`, row pitch lddx; a row with a negative target
 *            becomes 0, one with a target >= vocab NaN, any other with a g_loss
 *            of 0 becomes 0 whatever its lse
 */
q4_status q4_head_cross_entropy_backward(
    const void *x, int64_t ldx, int32_t dtype, int64_t M, int64_t vocab,
    int64_t K, const uint8_t *qw, const float *scales, int64_t group_size,
    int32_t nibble_order, const int64_t *targets, const float *lse,
    const float *g_loss, void *dx, int64_t lddx, void *workspace,
    size_t workspace_bytes, void *stream);

/* Bytes of workspace q4_head_cross_entropy_backward needs (0 for invalid
 * sizes). */
size_t q4_head_cross_entropy_backward_workspace_bytes(int32_t dtype, int64_t M,
                                                      int64_t vocab, int64_t K,
                                                      int64_t group_size);

#ifdef __cplusplus
}
#endif

#endif /* Q4EXPERTS_H */
