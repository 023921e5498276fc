/*
 * ffn_experts.h -- C ABI of routing to experts (MI355X / gfx950), part of the
 * same library as ffn_sparse.h: the router's scores and choice of experts, the
 * order of the rows by expert, the rows' way to the experts and back, and the
 * gradients of each. The products between are ffn_linear.h's, which takes the
 * offsets made here.
 *
 * Conventions are those of ffn_linear.h: device pointers allocated by the
 * caller, 16-byte aligned, row-major dense; calls are asynchronous on `stream`,
 * check their arguments before launching anything, write nothing on an error,
 * allocate nothing, keep no state and may be captured into a graph. A call
 * without rows does nothing but what is said below, and takes null pointers. An
 * output shares memory with an input only where that is said.
 * `dtype` is ffn_dtype (FFN_F32 or FFN_BF16); sums are held in fp32 or more and
 * made in a fixed order, so results are the same from run to run. m * top_k is
 * at most 2^31 - 2^16.
 */
#ifndef FFN_EXPERTS_H
#define FFN_EXPERTS_H

#include <stddef.h>
#include <stdint.h>

#include "ffn_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FFN_EXPERTS_ABI_VERSION 1
#define FFN_ROUTE_MAX_EXPERTS 256
#define FFN_ROUTE_MAX_TOP_K 16
#define FFN_ROUTE_MAX_GROUPS 32
#define FFN_ROWS_MAX_GROUPS 1024

typedef enum { FFN_ROUTE_SOFTMAX = 0, FFN_ROUTE_SIGMOID = 1 } ffn_route_score;

int32_t ffn_experts_abi_version(void);

/* The choice of top_k experts for each of m tokens, and their weights.
 *   logits  [m x experts] dtype; score is softmax or sigmoid (ffn_route_score):
 *           s = softmax(l) over the token's experts, or 1 / (1 + exp(-l))
 *   bias    NULL or [experts] fp32, finite: added to the scores for the choice
 *           alone (balancing the experts without a loss): v = s + bias
 *   groups, top_groups, group_best   experts stand in `groups` groups of equal
 *           size, one after the other; of these the top_groups best stay, by the
 *           sum of a group's group_best (1 or 2) largest v. groups = top_groups:
 *           all stay
 *   ids     [m x top_k] int32: the experts of the largest v in the groups that
 *           stay, largest first
 *   weights [m x top_k] fp32: scale * s of the chosen, or with renormalize = 1
 *           scale * s / (the sum of the token's chosen s); without the bias
 *   scores  NULL or [m x experts] fp32: s (for losses on all of them)
 * Equal values go to the lower index (of the group, and of the expert). Where
 * scores decide they are told apart in fp64 (nothing but its rounding, 2^-53 of a
 * score or of a group's sum, can confuse them), so that the choice is that of the
 * exact scores; without a bias experts stand in the order of their logits, and
 * so do groups with group_best = 1.
 * An expert whose logit is -inf is never chosen, and a group with no other is
 * never kept; where fewer than top_k experts are left, the last slots have id
 * -1 and weight 0, and a token without any has scores of 0. Zeros of both signs
 * are equal. A NaN counts as +inf, and whatever it enters is NaN (softmax: all of
 * the token's scores and weights, as with a logit of +inf; the ids are then any of
 * its experts).
 * 1 <= experts <= 256, 1 <= top_k <= min(16, experts), 1 <= groups <= 32, groups
 * divides experts, 1 <= top_groups <= groups, scale finite. */
ffn_status ffn_route_forward(const void *logits, int32_t dtype, int32_t m, int32_t experts, int32_t top_k,
                             int32_t score, const float *bias, int32_t groups, int32_t top_groups,
                             int32_t group_best, int32_t renormalize, float scale, float *weights, int32_t *ids,
                             float *scores, void *stream);

/* Gradient of <dweights, weights> + <dscores, scores> of the call above, with
 * its choice held fixed:
 *   ids       [m x top_k] as it gave them; slots whose id is no expert count for nothing
 *   dweights  [m x top_k] fp32; dscores NULL or [m x experts] fp32
 *   dlogits   [m x experts] dtype, written in full (may be logits itself) */
ffn_status ffn_route_backward(const void *logits, int32_t dtype, int32_t m, int32_t experts, int32_t top_k,
                              int32_t score, int32_t renormalize, float scale, const int32_t *ids,
                              const float *dweights, const float *dscores, void *dlogits, void *stream);

/* Bytes of workspace ffn_group_rows needs (0: none, or invalid). */
size_t ffn_group_rows_workspace_bytes(int32_t n, int32_t groups);

/* The order of n entries by group: entries of a group stay in their own order,
 * entries of no group (ids outside 0 .. groups - 1) come last.
 *   ids      [n] int32 (the experts of [m x top_k] slots, the adapters of m rows)
 *   offsets  [groups + 1]: group g has places offsets[g] .. offsets[g + 1] - 1,
 *            as ffn_linear.h takes them
 *   rows     NULL or [n]: the entry at each place
 *   slots    NULL or [n]: the place of each entry, -1 for entries of no group
 * With n = 0, offsets is cleared. 1 <= groups <= FFN_ROWS_MAX_GROUPS; n <= 2^24
 * (FFN_E_UNSUPPORTED above). Made for up to some hundred thousand entries: from a
 * million on the time grows with their square (2^20 of 256 groups 57 us, 2^24 4.8
 * ms). */
ffn_status ffn_group_rows(const int32_t *ids, int32_t n, int32_t groups, int32_t *offsets, int32_t *rows,
                          int32_t *slots, void *workspace, size_t workspace_bytes, void *stream);

/* The rows of m tokens to their places: y[slots[t, s]] = x[t].
 *   x       [m x d] dtype
 *   slots   [m x top_k] int32, different places; one outside 0 .. m * top_k - 1 has no row
 *   y       NULL or [m * top_k x d] dtype
 *   q, scale  NULL or the same rows in 8-bit blocks of 1 x 128 (ffn_linear.h):
 *           q [m * top_k x d], scale [ceil(d / 128) x m * top_k]
 * One of y and q at least. Rows that no slot names are left as they were. d:
 * multiple of 8, up to 2^22. 1 <= top_k <= 16. Each row of x is read once. */
ffn_status ffn_gather_forward(const void *x, int32_t dtype, int32_t m, int32_t d, const int32_t *slots, int32_t top_k,
                              void *y, uint8_t *q, float *scale, void *stream);

/* The experts' rows back to their tokens, summed in fp32 in slot order and
 * rounded once: out[t] = residual[t] + sum over s of weights[t, s] y[slots[t, s]].
 *   y        [m * top_k x d] dtype; slots as above: a slot without a row adds nothing
 *   weights  NULL (ones) or [m x top_k] fp32
 *   residual NULL or [m x d] dtype
 *   out      [m x d] dtype (may be residual itself)
 * Without weights also the gradient of ffn_gather_forward. */
ffn_status ffn_combine_forward(const void *y, int32_t dtype, int32_t m, int32_t d, const int32_t *slots, int32_t top_k,
                               const float *weights, const void *residual, void *out, void *stream);

/* Gradients of <dout, out> of the call above (that of the residual is dout):
 *   dy        NULL or [m * top_k x d] dtype: dy[slots[t, s]] = weights[t, s] dout[t];
 *             rows that no slot names are left as they were (may be y itself)
 *   dweights  NULL or [m x top_k] fp32: <dout[t], y[slots[t, s]]>, 0 for a slot without a row
 * One of them at least; y may be NULL without dweights. weights as above. */
ffn_status ffn_combine_backward(const void *y, int32_t dtype, int32_t m, int32_t d, const int32_t *slots, int32_t top_k,
                                const float *weights, const void *dout, void *dy, float *dweights, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FFN_EXPERTS_H */
