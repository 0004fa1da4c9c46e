/*
 * moe_train.h — the MoE layer's training step: token rows moved by expert and
 * back, the router's gradient, the experts' grouped products, the norms, gate
 * and residual of the block around the layer, each with its gradient; and
 * activations kept for the backward pass in 8 bits.  Conventions as in moe.h (status codes, caller-owned device
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
 *
 * Around the layer: moe_norm_rows gives the layer's input from the residual
 * stream, moe_block_out takes its output back into the stream (and gives the
 * next layer's input).  moe_block_out serves inference as well, on the float32
 * output of moe_layer_forward.
 *
 * Packed rows: rows [rows, cols] in 8 bits, for activations that wait for the
 * backward pass.  Blocks of 32 columns of a row share a power of two.  With
 * nb = (cols + 31) / 32:
 *   q      int8  [rows, 32 nb]  byte 4 (c % 8) + c / 8 of a block is its column c
 *   scale  uint8 [rows, nb]     E; a value is q 2^(E - 127)
 * The four columns c, c + 8, c + 16, c + 24 of a word are those that a thread
 * holds of a matrix fragment.  E is the least for which every |q| is at most
 * 127 (0 at least: values below 2^-128 become zero; 248 at most: a magnitude
 * above 127 2^121 becomes that); q is rounded to nearest, ties to even, so a
 * value is off by at most half of 2^(E - 127), 1/127 of its block's largest
 * magnitude.  A block with a value that is not finite has
 * E = 255: all its values read as NaN.  Bytes past the last column are zero.
 * What is read back is exact in bf16 and float32.  q is 16-byte aligned.
 *
 *   moe_experts_up_packed   as moe_experts_up, g and u packed
 *   moe_pack_rows           x [T, d] (one row a token; not x_perm), y_perm
 *   moe_combine_rows_grad_packed, moe_experts_down_grad_packed
 *   moe_unpack_rows         x_perm again, for moe_experts_up_grad
 * A slot then keeps d + 2 I bytes and their scales instead of 2 (2 d + 3 I).
 */
#ifndef MOE_GB300_TRAIN_H
#define MOE_GB300_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device workspace for the calls below with these dims (at most 16 MiB; 12 of it
 * hold the sums over the tokens of moe_norm_rows_grad and moe_block_out_grad, and
 * the other calls take a workspace without them).
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

/* ------------------------------------------------------------ the block around the layer
 * Norms are root mean square norms: rstd = (mean_j x_j^2 + eps)^-1/2 over a
 * row's d values, n_j = x_j rstd (weight_offset + w_j).  Squares whose sum
 * passes float32's range are summed again at a smaller scale; below it they are
 * lost beside an eps that is a normal number.  Long batches wait
 * for their rows inside the kernel.  A wait that gives up (about a second) makes
 * that row's results NaN, those of the rows that the same threads would have taken
 * after it, and the sums over the tokens, and gives MOE_ERR_TIMEOUT in the error
 * word of the gradients (moe_norm_rows and moe_block_out have none). */

/* The factor on the block's output before it joins the residual. */
typedef enum {
    MOE_GATE_NONE = 0,
    MOE_GATE_TOKEN = 1,    /* float32 [T] */
    MOE_GATE_CHANNEL = 2,  /* [d] of the layer's type */
    MOE_GATE_FULL = 3      /* [T, d] of the layer's type, contiguous */
} moe_block_gate;

/* eps > 0, finite; weight_offset (0, or 1 for weights that start from one) and
 * residual_scale finite; post_norm: whether the block's output is normed. */
typedef struct {
    float eps, weight_offset, residual_scale;
    int post_norm;
    int gate; /* moe_block_gate */
} moe_block;

/* n = x rstd (weight_offset + weight): the norm before a block.
 *   x, n [T, d] (n may be x); weight [d] of the layer's type (NULL = zeros:
 *   n = weight_offset x rstd); rstd [T] float32 (NULL = skip; kept for the
 *   gradient). */
moe_status moe_norm_rows(const moe_dims* dims, const void* x, int64_t ldx, const void* weight, float eps,
                         float weight_offset, void* n, int64_t ldn, float* rstd, void* stream);

/* Gradient of moe_norm_rows: with xn = x rstd and g = dn (weight_offset + weight),
 *   dx = add + rstd (g - xn mean_j(g xn))   (dx may be add or dn; add NULL = zero)
 *   dweight = sum_t dn xn                   (NULL = skip)
 * rstd as moe_norm_rows gave it.  gtype: the type of dweight [d], wtype or
 * float32; accumulate != 0 adds to what it holds (float32 only). */
moe_status moe_norm_rows_grad(const moe_dims* dims, const void* dn, int64_t lddn, const void* x, int64_t ldx,
                              const float* rstd, const void* weight, float weight_offset, const void* add,
                              int64_t ldadd, void* dx, int64_t lddx, void* dweight, moe_dtype gtype,
                              int accumulate, void* ws, size_t ws_bytes, void* stream);

/* The end of a block: its output y through the norm after it, the gate, the
 * residual scale and the residual, and the norm before the next block.
 *   p    = y a (weight_offset + w_post) with post_norm (a: y's rstd), else y
 *   out  = residual + residual_scale gate p
 *   next = out b (weight_offset + w_next)   (b: out's rstd, of out before its rounding)
 *   y [T, d] of type ytype (wtype, or float32); residual, out, next [T, d] (out
 *   may be residual; next NULL = no next norm); gate as block->gate says, NULL
 *   for MOE_GATE_NONE; w_post, w_next [d] (NULL = zeros; w_post only with
 *   post_norm, w_next only with next); rstd_post, rstd_next [T] float32 (NULL =
 *   skip; kept for the gradient). */
moe_status moe_block_out(const moe_dims* dims, const moe_block* block, const void* y, int64_t ldy,
                         moe_dtype ytype, const void* residual, int64_t ldr, const void* gate,
                         const void* w_post, const void* w_next, void* out, int64_t ldo, void* next,
                         int64_t ldn, float* rstd_post, float* rstd_next, void* stream);

/* Gradient of moe_block_out.  dout: the gradient of out by its other uses (NULL =
 * zero), dnext that of next (NULL = zero: the block has no next norm; one of the
 * two is needed); y, out, gate, w_post, w_next, rstd_post, rstd_next as in or
 * from the forward call (out, w_next, rstd_next with dnext; y and rstd_post
 * where dy, dgate or dw_post ask for them).  With xo = out b, yn = y a:
 *   D         = dout + b (g - xo mean(g xo)),  g = dnext (weight_offset + w_next)
 *   dresidual = D                                      (may be dout or dnext; NULL = skip)
 *   dgate     = residual_scale sum D p over the axis that the gate is spread on (NULL = skip)
 *   dy        = residual_scale D gate, with post_norm through the norm (type ytype; NULL = skip)
 *   dw_post   = residual_scale sum_t D gate yn,  dw_next = sum_t dnext xo   (NULL = skip)
 * dgate is float32 [T], of type gtype [d], or of the layer's type [T, d]; dw_post and
 * dw_next have type gtype, wtype or float32; accumulate != 0 adds to what those of
 * type gtype hold (float32 only). */
moe_status moe_block_out_grad(const moe_dims* dims, const moe_block* block, const void* dout, int64_t lddout,
                              const void* dnext, int64_t lddnext, const void* y, int64_t ldy,
                              moe_dtype ytype, const void* out, int64_t ldo, const void* gate,
                              const void* w_post, const void* w_next, const float* rstd_post,
                              const float* rstd_next, void* dresidual, int64_t lddr, void* dy, int64_t lddy,
                              void* dgate, void* dw_post, void* dw_next, moe_dtype gtype, int accumulate,
                              void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------ activations in 8 bits */

/* Bytes of q and scale for `rows` rows of `cols` values (packed rows, above). */
moe_status moe_packed_size(int64_t rows, int cols, size_t* q_bytes, size_t* scale_bytes);

/* x [rows, cols] of type xtype (row stride ldx in elements, 0 = cols) -> packed rows.
 * rows up to 2^24, cols up to 65536. */
moe_status moe_pack_rows(int64_t rows, int cols, const void* x, int64_t ldx, moe_dtype xtype, int8_t* q,
                         uint8_t* scale, void* stream);

/* Packed rows [src_rows, cols] back to values: out[i] = row index[i] / divisor
 * (index NULL: row i), i < rows, of type otype (row stride ldo in elements, 0 =
 * cols).  A negative index, or one whose row is not there, gives a row of zeros.
 * With moe_dispatch_rows' perm and divisor k, out is x_perm. */
moe_status moe_unpack_rows(int64_t src_rows, int cols, const int8_t* q, const uint8_t* scale,
                           const int32_t* index, int divisor, int64_t rows, void* out, int64_t ldo,
                           moe_dtype otype, void* stream);

/* moe_experts_up with g and u [T*k, I] packed from their float32 sums (h is that
 * of the sums too).  Rows of no expert pack to zeros. */
moe_status moe_experts_up_packed(const moe_dims* dims, const void* x_perm, const int32_t* expert_offsets,
                                 const void* w_gate, const void* w_up, int8_t* g_q, uint8_t* g_scale,
                                 int8_t* u_q, uint8_t* u_scale, void* h, void* ws, size_t ws_bytes,
                                 void* stream);

/* moe_experts_down_grad with g and u packed, and h = SiLU(g) (.) u of the packed
 * values formed anew: dg, du and h [T*k, I] are written, dw_down (NULL = skip)
 * is h^T dy of that h as it is rounded. */
moe_status moe_experts_down_grad_packed(const moe_dims* dims, const void* dy_perm, const int8_t* g_q,
                                        const uint8_t* g_scale, const int8_t* u_q, const uint8_t* u_scale,
                                        const int32_t* expert_offsets, const void* w_down, void* h, void* dg,
                                        void* du, void* dw_down, moe_dtype gtype, int accumulate, void* ws,
                                        size_t ws_bytes, void* stream);

/* moe_combine_rows_grad with y_perm [T*k, d] packed. */
moe_status moe_combine_rows_grad_packed(const moe_dims* dims, const void* dout, int64_t lddout,
                                        const int8_t* y_q, const uint8_t* y_scale, const float* gate,
                                        const int32_t* inv_perm, void* dy_perm, float* dgate, void* stream);

/* Which kernels the experts' products run for these dims (buffers 16-byte
 * aligned): "tc" (tcgen05) or "simt" (CUDA cores); "unsupported" for bad
 * dims.  No device work. */
const char* moe_experts_path(const moe_dims* dims);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_TRAIN_H */
