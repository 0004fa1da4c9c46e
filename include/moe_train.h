/*
 * moe_train.h — the MoE layer's training step: token rows moved by expert and
 * back, the router's gradient, and the experts' grouped products, each with
 * its gradient.  Conventions as in moe.h (status codes, caller-owned device
 * buffers, everything queued on the caller's stream, on the current device,
 * to which stream and buffers have to belong; device-detected errors
 * in the workspace's error word, read by moe_check()).
 *
 * A slot (t, s) is one of token t's k choices; its expert is
 * expert_idx[t * k + s].  moe_dispatch_rows sorts the slots by expert and
 * copies the token rows; moe_experts_up and moe_experts_down run the experts'
 * SwiGLU FFN on the grouped rows; moe_combine_rows brings the results back,
 * weighted by the gates.  Forward, then backward:
 *
 *   moe_route (or any router)      -> topk_idx, topk_gate, router_prob
 *   moe_dispatch_rows              -> x_perm, expert_offsets, perm, inv_perm
 *   moe_experts_up                 -> g, u, h = SiLU(g) (.) u
 *   moe_experts_down               -> y_perm
 *   moe_combine_rows               -> out = add + sum_s gate y
 *   moe_combine_rows_grad  (dout)  -> dy_perm, dgate
 *   moe_experts_down_grad          -> dg, du, dw_down
 *   moe_experts_up_grad            -> dx_perm, dw_gate, dw_up
 *   moe_gate_grad                  -> dlogits, balance loss
 *   moe_dispatch_rows_grad         -> dx
 *
 * dims (moe_dims) as in moe.h, with the limits of these calls: d and I of any
 * value from 1 to 65536, N <= 512, k <= 16, k <= N, T * k <= 2^24; n_shared, I_shared, r and
 * delta_max are not looked at.  Rows (x, y_perm, h, weights, their gradients)
 * have the layer's type wtype (bf16 or float32); gates, router probabilities
 * and logits' gradients are float32; indices int32.  Sums run in float32 in an
 * order that does not change from call to call; each output is rounded once.
 *
 * Row counts: the grouped tensors have T * k rows.  Expert e's rows are
 * expert_offsets[e] .. expert_offsets[e + 1]; rows from expert_offsets[N] on
 * belong to no expert.  Every output row there is written as zero.
 *
 * Row strides: tensors of token rows (x, dx, out, dout, add) take a row
 * stride in elements (0 = d), so that they may be part of a wider tensor.
 * Grouped tensors and weights are contiguous.
 *
 * The pages treat inference; the gradients here are those of their forward
 * formulas (router softmax and top-k, APEX §4.1; SwiGLU experts, FloE method
 * §1; gate-weighted sum, SPICE).
 */
#ifndef MOE_GB300_TRAIN_H
#define MOE_GB300_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device workspace for the calls below with these dims (at most 16 MiB).
 * Zero-fill it once before first use.  Its error word sits where moe_check()
 * looks for it. */
moe_status moe_train_workspace_size(const moe_dims* dims, size_t* bytes);

/* Sort the T * k slots by expert, stable in slot order, and copy the rows.
 *   x [T, d] (row stride ldx); expert_idx [T, k]: the expert of each slot, a
 *   negative value = no expert.  capacity > 0: an expert takes its first
 *   `capacity` slots, the rest of its slots have no expert; 0 = no limit.
 *   x_perm [T*k, d]: row pos = x[slot / k] of the slot at pos, zero past the
 *   last expert's rows.  expert_offsets [N+1]; perm [T*k]: the slot at pos,
 *   -1 past the last expert's rows; inv_perm [T*k]: the slot's pos, or, for a
 *   slot without an expert, -2 - (its zero row in x_perm).
 * An index >= N sets MOE_ERR_DEVICE_INDEX in the error word and counts as no
 * expert.  Errors: INVALID_ARG (NULL or misaligned buffer, capacity < 0,
 * ldx < d), UNSUPPORTED (dims), CAPACITY (workspace), CUDA. */
moe_status moe_dispatch_rows(const moe_dims* dims, const void* x, int64_t ldx, const int32_t* expert_idx,
                             int capacity, void* x_perm, int32_t* expert_offsets, int32_t* perm,
                             int32_t* inv_perm, void* ws, size_t ws_bytes, void* stream);

/* dx[t] = add[t] + sum over token t's slots with an expert of
 * dx_perm[inv_perm[t, s]].  add may be NULL (zero) and may be dx itself. */
moe_status moe_dispatch_rows_grad(const moe_dims* dims, const void* dx_perm, const int32_t* inv_perm,
                                  const void* add, int64_t ldadd, void* dx, int64_t lddx, void* stream);

/* out[t] = add[t] + sum over token t's slots with an expert of
 * gate[t, s] * y_perm[inv_perm[t, s]].  gate NULL = 1; add may be NULL (zero)
 * and may be out itself (the shared experts' output, a residual).  A token
 * none of whose slots has an expert gets add[t].  The inv_perm of moe_permute
 * serves too (-1 = no row); an entry >= T*k counts as no row. */
moe_status moe_combine_rows(const moe_dims* dims, const void* y_perm, const float* gate,
                            const int32_t* inv_perm, const void* add, int64_t ldadd, void* out,
                            int64_t ldout, void* stream);

/* Gradient of moe_combine_rows:
 *   dy_perm[inv_perm[t, s]] = gate[t, s] * dout[t] (NULL = skip), zero in the
 *   rows past the last expert's (with moe_permute's inv_perm, whose -1 names no
 *   row, those stay unwritten); dgate[t, s] = <dout[t], y_perm[inv_perm[t, s]]>,
 *   zero for a slot without an expert (NULL = skip; needs y_perm).  gate NULL
 *   = 1.  add's gradient is dout. */
moe_status moe_combine_rows_grad(const moe_dims* dims, const void* dout, int64_t lddout, const void* y_perm,
                                 const float* gate, const int32_t* inv_perm, void* dy_perm, float* dgate,
                                 void* stream);

/* The router's gradient: gates back through the top-k and the softmax.
 *   router_prob [T, N] = p (softmax of the logits, moe_route's output);
 *   topk_idx [T, k] (negative = no expert); dgate [T, k].
 *   dims->renorm_topk 0: gate_s = p_{i_s}; 1: gate_s = p_{i_s} / sum over the
 *   token's slots.  balance = c >= 0 adds the load-balance loss
 *   c N sum_e f_e P_e, f_e = the share of the T k slots that chose e (a
 *   constant in the gradient), P_e = the mean over tokens of p_e.
 *   dlogits [T, N]; balance_loss [1] (NULL = skip).  The sum of a token's
 *   gates being zero gives its slots no gradient. */
moe_status moe_gate_grad(const moe_dims* dims, const float* router_prob, const int32_t* topk_idx,
                         const float* dgate, float balance, float* dlogits, float* balance_loss, void* ws,
                         size_t ws_bytes, void* stream);

/* The experts' up products on the grouped rows: per expert e and its rows,
 *   g = x Wg_e^T, u = x Wu_e^T, h = SiLU(g) (.) u.
 *   x_perm [T*k, d]; w_gate, w_up [N, I, d]; g, u (both or neither NULL: kept
 *   for the gradient) and h: [T*k, I].  Tensor cores when wtype is bf16, d and
 *   I are multiples of 8 from 64 on and every matrix is 16-byte aligned; CUDA
 *   cores in float32 arithmetic otherwise.  moe_experts_path names the choice. */
moe_status moe_experts_up(const moe_dims* dims, const void* x_perm, const int32_t* expert_offsets,
                          const void* w_gate, const void* w_up, void* g, void* u, void* h, void* ws,
                          size_t ws_bytes, void* stream);

/* Gradient of the up products: dx_perm = dg Wg_e + du Wu_e (NULL = skip),
 * dw_gate[e] = dg^T x, dw_up[e] = du^T x over expert e's rows (both or neither
 * NULL; an expert without rows gets zeros).  gtype: the type of dw_gate and
 * dw_up [N, I, d], wtype or float32.  accumulate != 0 adds to what they hold
 * (float32 only, UNSUPPORTED otherwise; without them it says nothing). */
moe_status moe_experts_up_grad(const moe_dims* dims, const void* dg, const void* du, const void* x_perm,
                               const int32_t* expert_offsets, const void* w_gate, const void* w_up,
                               void* dx_perm, void* dw_gate, void* dw_up, moe_dtype gtype, int accumulate,
                               void* ws, size_t ws_bytes, void* stream);

/* The experts' down product: y_perm = h Wd_e; h [T*k, I], w_down [N, I, d],
 * y_perm [T*k, d]. */
moe_status moe_experts_down(const moe_dims* dims, const void* h, const int32_t* expert_offsets,
                            const void* w_down, void* y_perm, void* ws, size_t ws_bytes, void* stream);

/* Gradient of the down product, taken through h = SiLU(g) (.) u: with
 * dh = dy Wd_e^T (never rounded) and s = sigmoid(g),
 *   dg = dh u s (1 + g (1 - s)), du = dh g s   (both or neither NULL),
 *   dw_down[e] = h^T dy over expert e's rows (NULL = skip; an expert without
 *   rows gets zeros).  gtype, accumulate as in moe_experts_up_grad. */
moe_status moe_experts_down_grad(const moe_dims* dims, const void* dy_perm, const void* h, const void* g,
                                 const void* u, const int32_t* expert_offsets, const void* w_down, void* dg,
                                 void* du, void* dw_down, moe_dtype gtype, int accumulate, void* ws,
                                 size_t ws_bytes, void* stream);

/* Which kernels the experts' products run for these dims (buffers 16-byte
 * aligned): "tc" (tcgen05) or "simt" (CUDA cores); "unsupported" for bad
 * dims.  No device work. */
const char* moe_experts_path(const moe_dims* dims);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_TRAIN_H */
