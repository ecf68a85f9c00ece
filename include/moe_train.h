/*
 * moe_train.h -- the router's training operators of libmoe_b200 (C ABI): the load-balance
 * loss with the per-expert counts, and the gradient of the routing weights and of that
 * loss with respect to the router logits.  Types, status codes and conventions are those
 * of moe.h.
 *
 * Definitions, for logits l [T, E], l' = fp32(l) + fp32(router_bias) and a routing
 * idx [T, k] (moe_route's, or any; an index outside [0, E) is a slot without an expert):
 *   p[t, e]  = softmax_e(l'[t])            (MOE_SCORE_SOFTMAX)
 *            = sigma(l'[t, e]) / sum_e sigma(l'[t, e])  (MOE_SCORE_SIGMOID)
 *              and 0 throughout for a row whose logits l' are all -inf (sigmoid: all below
 *              -700, as masks of the type's lowest value are);
 *   sequence b holds the tokens seq_offsets[b] .. seq_offsets[b + 1] - 1, n_b of them
 *              (NULL: one sequence of all T tokens; tokens outside every sequence are
 *              padding and enter nothing);
 *   counts[b, e] = the slots (t, j) of sequence b with idx[t, j] == e;
 *   loss = coef / B' sum_b E / (k n_b^2) sum_e counts[b, e] sum_{t in b} p[t, e],
 *              B' = the sequences with n_b > 0 (loss 0 if none): 1 times coef when every
 *              expert gets the same share.
 * The gradient takes the counts as constants (they are integers).
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace moe_balance_loss needs for B sequences (0 if the arguments are
 * invalid; moe_last_error() then says why). */
MOE_API size_t moe_balance_workspace_size(const moe_shape *shape, const moe_options *opts, int64_t B);

/* The balance loss and the counts.  Of the shape T, E, k and logit_dtype are used, of the
 * options score.
 *   logits       [T, E] logit_dtype
 *   router_bias  [E] logit_dtype, optional
 *   idx          [T, k] int32
 *   seq_offsets  [B + 1] int32, not decreasing, in 0 .. T; NULL with B == 1
 *   counts       [B, E] int32, output
 *   loss         [1] fp32, output
 *   workspace    256-byte aligned, used by this call alone until it completes
 * Sums are fp32 per block of tokens and double across blocks, in a fixed order: results
 * are bitwise reproducible.  Errors: MOE_ERR_NULL / SHAPE / ARG / ALIGN / WORKSPACE before
 * any launch, MOE_ERR_CUDA if a launch fails. */
MOE_API int moe_balance_loss(const moe_shape *shape, const moe_options *opts, const void *logits,
                             const void *router_bias, const int32_t *idx, const int32_t *seq_offsets, int64_t B,
                             float coef, int32_t *counts, float *loss, void *workspace, size_t workspace_bytes,
                             void *stream);

/* The gradient with respect to the logits (and, summed over the tokens, to router_bias) of
 *   sum_{t, j} dw[t, j] w[t, j] + dloss * loss
 * with w moe_route's weights of the slots idx (score, renormalize, routed_scale: w_j = S s_j,
 * or S s_j / max(sum_j s_j, 2^-14); the clamped sum is a constant, a sum equal to the clamp
 * is not clamped) and loss as above for the given counts.
 *   dw       [T, k] fp32, or NULL (no routing part)
 *   counts   [B, E] int32, moe_balance_loss's, or NULL (no balance part: seq_offsets, B,
 *            coef and dloss are not used).  Counts summed over data-parallel ranks of n_b
 *            tokens each give the gradient of the global loss with coef / ranks.
 *   dloss    [1] fp32 on the device, or NULL (1)
 *   dlogits  [T, E] logit_dtype, output: every element is written; computed in fp32 and
 *            rounded once
 * At least one of dw and counts is given.  dw of a slot without an expert is not used.
 * A row of which nothing enters (a token outside every sequence, or no counts, without a
 * slot that has an expert or without dw) gives 0, whatever its logits.  Else, with
 * MOE_SCORE_SOFTMAX a row with a NaN or +inf logit gives NaN; with MOE_SCORE_SIGMOID a NaN
 * logit gives NaN where the formulas depend on it.  Errors as above; T == 0 is a no-op. */
MOE_API int moe_router_backward(const moe_shape *shape, const moe_options *opts, const void *logits,
                                const void *router_bias, const int32_t *idx, const float *dw, const int32_t *counts,
                                const int32_t *seq_offsets, int64_t B, float coef, const float *dloss, void *dlogits,
                                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */
