/*
 * libmoe_epi — the steps around the routed experts: the order of the rows, the
 * moves of the rows with their gradients, and the experts' products in 8-bit
 * integers. Status codes, dtype codes and the common contract (memory owned by
 * the caller, nothing allocated, nothing kept between calls, no
 * synchronisation, capture into HIP graphs, arguments checked on the host
 * before any launch, no output overlapping an input or another output) are
 * those of moe_epi.h.
 *
 * A slot is one choice of one token: slot t * top_k + j is choice j of token
 * t. A row is one slot that an expert of this GPU takes; rows are grouped by
 * expert. moe_sort_fwd gives the three tensors that connect them:
 *   offs    [experts] int32          rows up to and with expert e (cumulative)
 *   row_of  [tokens, top_k] int32    the row of a slot, -1 if it has none
 *   slot_of [tokens * top_k] int32   the slot of a row, -1 past the last row
 * Every call that takes an index tensor checks each index on the device and
 * leaves out those that are out of range, so a wrong index gives wrong values
 * and never an access outside the tensors.
 */
#ifndef MOE_ROUTED_H
#define MOE_ROUTED_H

#include "moe_epi.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Order of the rows: a stable counting sort of the slots by local expert.
 * The experts of this GPU are [first_expert, first_expert + experts); a slot
 * whose expert is not one of them has no row. Rows are ordered by expert and,
 * within an expert, by slot (ascending), which makes the order unique: the
 * results are the same in every run.
 *   offs[e]    = number of slots whose expert is in [first_expert, first_expert + e]
 *   row_of[s]  = the row of slot s, or -1
 *   slot_of[r] = the slot of row r for r < offs[experts - 1], else -1
 *   expert_of  [tokens, top_k] int32 or int64 (id_bytes 4 or 8)   in
 *   offs       [experts] int32                                    out
 *   row_of     [tokens, top_k] int32                              out
 *   slot_of    [tokens * top_k] int32                             out
 *   workspace  moe_sort_workspace_bytes(tokens, top_k, experts) bytes of device
 *              memory, 4-byte aligned, contents lost; may be NULL if that is 0
 * experts in [1, 1024], top_k in [1, 1024], tokens * top_k <= INT32_MAX
 * (MOE_EPI_ERR_BAD_SHAPE otherwise, also for a workspace that is too small);
 * an id_bytes other than 4 or 8 returns MOE_EPI_ERR_BAD_DTYPE. tokens == 0 is
 * valid: offs is then all 0.
 */
int moe_sort_fwd(const void *expert_of, int id_bytes, int64_t first_expert, int32_t *offs, int32_t *row_of,
                 int32_t *slot_of, void *workspace, int64_t workspace_bytes, int64_t tokens, int64_t top_k,
                 int64_t experts, void *stream);

/* Bytes of workspace that moe_sort_fwd needs; -1 for sizes that it refuses. */
int64_t moe_sort_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts);

/*
 * Dispatch: the tokens' rows in expert order, out[r, :] = x[slot_of[r] / top_k, :]
 * (bits copied). A row whose slot is outside [0, tokens * top_k) is set to +0:
 * every element of out is written.
 *   x       [tokens, hidden] of dtype     in (may be NULL if tokens == 0)
 *   slot_of [rows] int32                  in (the first rows entries of moe_sort_fwd's)
 *   out     [rows, hidden] of dtype       out
 * Any hidden >= 1; pointers aligned to the element. 16-byte aligned tensors
 * with a row of whole 16-byte pieces move fastest, others by vectors at the
 * element's alignment.
 */
int moe_dispatch_fwd(const void *x, int dtype, const int32_t *slot_of, void *out, int64_t rows, int64_t tokens,
                     int64_t top_k, int64_t hidden, void *stream);

/*
 * Gradient of the dispatch: grad_x[t, :] = sum_j grad_out[row_of[t, j], :] over
 * the slots whose row is in [0, rows), float32 additions in ascending slot
 * order from +0, rounded once to dtype. Every element of grad_x is written.
 *   grad_out [rows, hidden] of dtype      in (may be NULL if rows == 0)
 *   row_of   [tokens, top_k] int32        in
 *   grad_x   [tokens, hidden] of dtype    out
 */
int moe_dispatch_bwd(const void *grad_out, int dtype, const int32_t *row_of, void *grad_x, int64_t rows,
                     int64_t tokens, int64_t top_k, int64_t hidden, void *stream);

/*
 * Weighted combine: out[t, :] = sum_j weights[t, j] * expert_out[row_of[t, j], :]
 * over the slots whose row is in [0, rows): one float32 fused multiply-add per
 * slot, in ascending slot order from +0, rounded once to out_dtype. Every
 * element of out is written; a token without rows gets +0. The weight of a
 * slot without a row is not used (it may be NaN).
 *   expert_out [rows, hidden] of eo_dtype   in (may be NULL if rows == 0)
 *   row_of     [tokens, top_k] int32        in
 *   weights    [tokens, top_k] float32      in
 *   out        [tokens, hidden]             out, of eo_dtype or float32
 *              (another out_dtype returns MOE_EPI_ERR_BAD_DTYPE)
 */
int moe_combine_weighted_fwd(const void *expert_out, int eo_dtype, const int32_t *row_of, const float *weights,
                             void *out, int out_dtype, int64_t rows, int64_t tokens, int64_t top_k, int64_t hidden,
                             void *stream);

/*
 * Gradients of the weighted combine, in one pass over grad_out and expert_out:
 *   grad_expert_out[row_of[t, j], :] = round(weights[t, j] * grad_out[t, :])
 *   grad_weights[t, j] = sum_h grad_out[t, h] * expert_out[row_of[t, j], h]
 * (float32, a fixed order), and grad_weights[t, j] = +0 for a slot without a
 * row. A row that no slot refers to is not written. Each row belongs to at
 * most one slot, as moe_sort_fwd gives them; if two slots name one row, its
 * gradient is that of either.
 *   grad_out        [tokens, hidden] of go_dtype (eo_dtype or float32)   in
 *   expert_out      [rows, hidden] of eo_dtype   in; may be NULL if grad_weights is NULL
 *   row_of          [tokens, top_k] int32        in
 *   weights         [tokens, top_k] float32      in
 *   grad_expert_out [rows, hidden] of eo_dtype   out
 *   grad_weights    [tokens, top_k] float32      out; may be NULL (not formed then)
 */
int moe_combine_weighted_bwd(const void *grad_out, int go_dtype, const void *expert_out, int eo_dtype,
                             const int32_t *row_of, const float *weights, void *grad_expert_out,
                             float *grad_weights, int64_t rows, int64_t tokens, int64_t top_k, int64_t hidden,
                             void *stream);

/*
 * Rows to 8-bit integers with one scale each:
 *   scale[r] = max_c |x[r, c]| / 127,  q[r, c] = rint(127 * x[r, c] / max_c |x[r, c]|)
 * in float32, ties to even, so that x is about q * scale. A row of zeros has
 * scale 0 and q 0. A row that holds an infinity or a NaN has scale NaN and
 * q 0: every product with it is NaN.
 *   x     [rows, cols] of dtype      in
 *   q     [rows, cols] int8          out
 *   scale [rows] float32             out
 * Any cols >= 1.
 */
int quantize_rows_int8_fwd(const void *x, int dtype, int8_t *q, float *scale, int64_t rows, int64_t cols,
                           void *stream);

/*
 * gate_up grouped product in 8-bit integers with the clamped SwiGLU epilogue.
 * Rows of expert e are [start_e, end_e) as in grouped_gate_up_swiglu_fwd, with
 * `rows` in the place of its tokens. For row r of expert e, u = slot_of[r] / top_k:
 *   gate[j] = float(sum_h a[u, h] * w_gate[e, j, h]) * a_scale[u] * w_gate_scale[e, j]
 *   up[j]   = float(sum_h a[u, h] * w_up[e, j, h])   * a_scale[u] * w_up_scale[e, j]
 *   y[r, j] = bf16( silu(min(gate[j], limit)) * clamp(up[j], -limit, limit) * probs[r] )
 * The sums are exact 32-bit integers (a hidden below 131072 keeps them so), the
 * rest is float32, rounded once. slot_of == NULL: u = r, tokens == rows, top_k == 1.
 * A row whose slot is outside [0, tokens * top_k) gives y = 0 * probs[r]. Rows
 * at or past the last end are not written. `rows` is what the tensors hold; how
 * many of them there are stands in offs, on the device, which the host does not
 * read. The results do not depend on rows beyond that, the time may: the kernel
 * is chosen by rows / experts, so tensors several times larger than the rows
 * they have get one made for more rows.
 *   a            [tokens, hidden] int8             in (may be NULL if tokens == 0)
 *   a_scale      [tokens] float32                  in (may be NULL if tokens == 0)
 *   slot_of      [rows] int32 or NULL              in
 *   w_gate, w_up [experts, inter, hidden] int8     in
 *   w_*_scale    [experts, inter] float32          in
 *   offs         [experts] int32, device memory    in
 *   probs        [rows] float32, or NULL for 1     in
 *   y            [rows, inter] bf16                out
 * hidden a multiple of 16 below 131072, inter a multiple of 8, rows at most
 * INT32_MAX (MOE_EPI_ERR_BAD_SHAPE otherwise); a, w_gate, w_up, y 16-byte
 * aligned, the rest 4-byte aligned (MOE_EPI_ERR_MISALIGNED); limit finite and
 * > 0 (MOE_EPI_ERR_BAD_LIMIT).
 */
int grouped_gate_up_swiglu_int8_fwd(const int8_t *a, const float *a_scale, const int32_t *slot_of,
                                    const int8_t *w_gate, const float *w_gate_scale, const int8_t *w_up,
                                    const float *w_up_scale, const int32_t *offs, const float *probs, uint16_t *y,
                                    int64_t rows, int64_t tokens, int64_t top_k, int64_t hidden, int64_t inter,
                                    int64_t experts, float limit, void *stream);

/*
 * Down grouped product in 8-bit integers with the router-weight multiply. For
 * row r of expert e:
 *   out[r, n] = out_dtype( float(sum_i h[r, i] * w_down[e, n, i]) * h_scale[r] * w_down_scale[e, n] * probs[r] )
 *   h            [rows, inter] int8                in
 *   h_scale      [rows] float32                    in
 *   w_down       [experts, hidden, inter] int8     in
 *   w_down_scale [experts, hidden] float32         in
 *   offs         [experts] int32, device memory    in
 *   probs        [rows] float32, or NULL for 1     in
 *   out          [rows, hidden] of out_dtype (MOE_EPI_BF16 or MOE_EPI_F32)   out
 * inter a multiple of 16 below 131072, hidden a multiple of 8; alignment and
 * the rest as above.
 */
int grouped_down_router_int8_fwd(const int8_t *h, const float *h_scale, const int8_t *w_down,
                                 const float *w_down_scale, const int32_t *offs, const float *probs, void *out,
                                 int out_dtype, int64_t rows, int64_t inter, int64_t hidden, int64_t experts,
                                 void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTED_H */
