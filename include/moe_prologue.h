/*
 * libmoe_epi — the steps before the routed experts: the norm that joins the
 * residual stream, the router's product, and the choice of each token's
 * experts, with their gradients. Status codes, dtype codes and the common
 * contract (memory owned by the caller, nothing allocated, nothing kept between
 * calls, no synchronisation, capture into HIP graphs, arguments checked on the
 * host before any launch, no output overlapping an input or another output
 * unless a call says so) are those of moe_epi.h. Sums are float32 in a fixed
 * order: the results are the same in every run.
 *
 * A workspace is device memory of the caller, 16-byte aligned, whose contents
 * are lost. Calls that may run at the same time (two streams, two captured
 * graphs) each need their own.
 */
#ifndef MOE_PROLOGUE_H
#define MOE_PROLOGUE_H

#include "moe_epi.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a token's scores come from its logits, and what a group of experts counts for. */
typedef enum moe_epi_score { MOE_EPI_SOFTMAX = 0, MOE_EPI_SIGMOID = 1 } moe_epi_score;
typedef enum moe_epi_group_score { MOE_EPI_GROUP_MAX = 0, MOE_EPI_GROUP_TOP2 = 1 } moe_epi_group_score;

/*
 * Root-mean-square norm of the rows of x, or of the residual stream with x added:
 *   h = round(x + residual)                (x where residual is NULL)
 *   n = 1 / sqrt(mean(h^2) + eps)          (h as stored, float32)
 *   y = h * n * weight                     (float32)
 *   residual_out = h, out = round(y), rstd = n
 *   scale = max|y| / 127, q = rint(127 y / max|y|)     (as quantize_rows_int8_fwd, of the unrounded y)
 * A row of zeros in y has scale 0 and q 0; a row with an infinity or a NaN in y
 * has scale NaN and q 0. The sum of squares is float32: rows whose squares
 * overflow it have n = 0, as 1 / sqrt(inf) is, and squares below its range count
 * as 0.
 *   x            [rows, cols] of dtype               in
 *   residual     [rows, cols] of dtype, or NULL      in
 *   weight       [cols] of w_dtype (dtype or float32)  in
 *   out          [rows, cols] of dtype, or NULL if q is given   out
 *   residual_out [rows, cols] of dtype, or NULL      out; may be residual itself
 *                (the stream updated in place); only with a residual
 *   q, scale     [rows, cols] int8 and [rows] float32, or both NULL   out
 *   rstd         [rows] float32, or NULL             out (for the gradient)
 * eps finite and >= 0 (MOE_EPI_ERR_BAD_LIMIT otherwise). Any cols >= 1.
 */
int rms_norm_fwd(const void *x, const void *residual, int dtype, const void *weight, int w_dtype, float eps, void *out,
                 void *residual_out, int8_t *q, float *scale, float *rstd, int64_t rows, int64_t cols, void *stream);

/*
 * Gradients of the norm, with a = h * rstd and g = grad_out * weight:
 *   grad_x[r]   = rstd[r] * (g - a * mean(g * a)) + grad_residual[r]
 *   grad_weight = sum_r grad_out[r] * a[r]
 * grad_x is the gradient of x and that of residual. Every element of both is
 * written (zeros in grad_weight where there are no rows).
 *   grad_out      [rows, cols] of dtype              in
 *   h             [rows, cols] of dtype              in (residual_out, or x where there was no residual)
 *   weight        [cols] of w_dtype (dtype or float32)  in
 *   rstd          [rows] float32                     in
 *   grad_residual [rows, cols] of dtype, or NULL     in (the gradient of residual_out)
 *   grad_x        [rows, cols] of dtype              out
 *   grad_weight   [cols] of w_dtype, or NULL         out
 *   workspace     rms_norm_bwd_workspace_bytes(rows, cols) bytes; may be NULL if grad_weight is
 */
int rms_norm_bwd(const void *grad_out, const void *h, int dtype, const void *weight, int w_dtype, const float *rstd,
                 const void *grad_residual, void *grad_x, void *grad_weight, void *workspace, int64_t workspace_bytes,
                 int64_t rows, int64_t cols, void *stream);

/* Bytes of workspace that rms_norm_bwd needs; -1 for sizes that it refuses. */
int64_t rms_norm_bwd_workspace_bytes(int64_t rows, int64_t cols);

/*
 * The router's product: logits[t, e] = sum_h x[t, h] * weight[e, h], products
 * of all bits of both (of two float32 factors up to 2^-23 of the product is left
 * out), float32 sums. x and weight of one 16-bit type follow IEEE arithmetic; where
 * one of them is float32, a row of x or of weight that holds an infinity or a NaN
 * gives NaN or an infinity, and a float32 factor is taken to 2^-134 (all bits of it
 * from 2^-110 on). The order of a sum depends on the sizes of the call, so a token's
 * logits may differ in their last bits in calls of other sizes.
 *   x         [tokens, hidden] of dtype                       in
 *   weight    [experts, hidden] of w_dtype (dtype or float32) in
 *   logits    [tokens, experts] float32                       out
 *   workspace moe_router_logits_workspace_bytes(tokens, hidden, experts) bytes; may be NULL if that is 0
 * experts in [1, 1024], hidden in [1, 2^24], tokens <= INT32_MAX.
 */
int moe_router_logits_fwd(const void *x, int dtype, const void *weight, int w_dtype, float *logits, void *workspace,
                          int64_t workspace_bytes, int64_t tokens, int64_t hidden, int64_t experts, void *stream);

/* Bytes of workspace that moe_router_logits_fwd needs; -1 for sizes that it refuses. */
int64_t moe_router_logits_workspace_bytes(int64_t tokens, int64_t hidden, int64_t experts);

/*
 * Gradients of the router's product:
 *   grad_x[t, h]      = sum_e grad_logits[t, e] * weight[e, h]
 *   grad_weight[e, h] = sum_t grad_logits[t, e] * x[t, h]
 * (products as in the forward call, float32 sums, rounded once). Every element is written.
 * A sum with an infinity or a NaN among its factors is NaN or an infinity, also
 * where IEEE arithmetic has an infinity, and no other sum is.
 *   grad_logits [tokens, experts] float32                       in
 *   x           [tokens, hidden] of dtype; may be NULL if grad_weight is           in
 *   weight      [experts, hidden] of w_dtype (dtype or float32); may be NULL if grad_x is   in
 *   grad_x      [tokens, hidden] of dtype, or NULL              out
 *   grad_weight [experts, hidden] of w_dtype, or NULL           out (not both NULL)
 *   workspace   moe_router_logits_bwd_workspace_bytes(tokens, hidden, experts) bytes; may be
 *               NULL if that is 0 or grad_weight is NULL
 * Sizes as in the forward call.
 */
int moe_router_logits_bwd(const float *grad_logits, const void *x, int dtype, const void *weight, int w_dtype,
                          void *grad_x, void *grad_weight, void *workspace, int64_t workspace_bytes, int64_t tokens,
                          int64_t hidden, int64_t experts, void *stream);

/* Bytes of workspace that moe_router_logits_bwd needs for a grad_weight; -1 for sizes that it refuses. */
int64_t moe_router_logits_bwd_workspace_bytes(int64_t tokens, int64_t hidden, int64_t experts);

/*
 * Choice of each token's experts, and the weights of the chosen:
 *   s = softmax(logits[t]) or sigmoid(logits[t]),  c = s + bias
 *   the experts are `groups` groups of equal size, one after the other; a group counts for its largest c
 *   (MOE_EPI_GROUP_MAX) or for the sum of its two largest (MOE_EPI_GROUP_TOP2); the top_groups best stay
 *   ids[t]     = the top_k experts of those groups with the largest c, in descending order
 *   weights[t] = scale * s[ids[t]], over their sum where renormalise is not 0
 * Ties go to the lowest index, of groups and of experts. Without a bias the
 * order is that of the logits (GROUP_TOP2: of the groups' sums of s); with one
 * it is that of c in 64 bits. The bias is for the choice alone: it is not in
 * the weights. Weights are float32; renormalised ones do not lose experts
 * whose scores underflow.
 * An expert with a logit or bias of -inf, or a NaN, is not chosen: where fewer
 * than top_k remain, the last ids are -1 (which moe_sort_fwd leaves out) with
 * weight 0. A token with a NaN logit, or under softmax with one of +inf, has
 * weights NaN; its ids are still different experts, or -1.
 *   logits  [tokens, experts] of dtype            in
 *   bias    [experts] float32, or NULL            in
 *   ids     [tokens, top_k] int32                 out
 *   weights [tokens, top_k] float32               out
 * experts in [1, 1024]; groups in [1, 64] and a divisor of experts (at least
 * two experts a group for GROUP_TOP2, where groups > 1); top_groups in [1,
 * groups]; top_k in [1, 64], at most the experts of top_groups groups; tokens
 * <= INT32_MAX. An unknown score or group_score is MOE_EPI_ERR_BAD_DTYPE; scale
 * finite (MOE_EPI_ERR_BAD_LIMIT).
 */
int moe_route_fwd(const void *logits, int dtype, const float *bias, int32_t *ids, float *weights, int64_t tokens,
                  int64_t experts, int64_t top_k, int64_t groups, int64_t top_groups, int score, int group_score,
                  int renormalise, float scale, void *stream);

/*
 * Gradient of the weights' choice with respect to the logits, the ids being
 * fixed. With u[j] = scale * grad_weights[t, j] for the slots whose id is an
 * expert, s as above and v the renormalised weights without scale:
 *   softmax:               grad_logits[e] = s[e] * (sum_{j: ids[j] = e} u[j] - sum_j u[j] s[ids[j]])
 *   softmax, renormalised: grad_logits[ids[j]] = v[j] * (u[j] - sum_i u[i] v[i])
 *   sigmoid:               grad_logits[ids[j]] = u[j] s (1 - s)
 *   sigmoid, renormalised: grad_logits[ids[j]] = (1 - s) v[j] * (u[j] - sum_i u[i] v[i])
 * and 0 for the other experts; slots with the same id add up. A slot whose id
 * is no expert has no part. Every element is written.
 *   grad_weights [tokens, top_k] float32       in
 *   logits       [tokens, experts] of dtype    in
 *   ids          [tokens, top_k] int32         in
 *   grad_logits  [tokens, experts] of dtype    out
 * Sizes as above.
 */
int moe_route_bwd(const float *grad_weights, const void *logits, int dtype, const int32_t *ids, void *grad_logits,
                  int64_t tokens, int64_t experts, int64_t top_k, int score, int renormalise, float scale,
                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PROLOGUE_H */
