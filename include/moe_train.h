/*
 * moe_train.h -- the training side of libmoe's C ABI: what runs backward
 * through one MoE layer whose experts stay quantized (their codes are frozen;
 * the router and whatever precedes the layer are trained).
 *
 *   forward:   moe_route_topk .. moe_combine (moe.h), then
 *              moe_act_pack8 (the layer's input kept in 8 bits) and
 *              moe_balance_loss (per-expert counts, balance and z losses)
 *   backward:  moe_expert_ffn_backward (recomputes the experts from the
 *              8-bit checkpoint; gradients of the input and of the gates),
 *              moe_route_backward (gradient of the router's logits) and
 *              moe_router_backward (gradients of the router's weights, and
 *              the router's share of the input's gradient)
 *
 * The conventions of moe.h hold for every call here: asynchronous on the
 * caller's stream, arguments checked on the host before anything is launched,
 * status codes and moe_last_error(), device pointers 16-byte aligned unless
 * stated otherwise, all memory owned by the caller, problems met on the device
 * reported in the device error word.  No call keeps anything between calls;
 * results do not depend on scheduling (no floating-point atomics).  The waits
 * inside the tensor-core kernels end after a second (the test hook
 * MOE_HOOK_WAIT_LIMIT_NS limits these too) with MOE_DEVERR_TIMEOUT.  Two calls
 * that overlap on the GPU must not share a workspace, which is scratch only:
 * it needs no initial contents.
 */
#ifndef MOE_TRAIN_H_
#define MOE_TRAIN_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation given as an 8-bit checkpoint (moe_act_pack8): codes, with their
 * scales in a second pointer.  Accepted where a call says so. */
#define MOE_Q8 2

/* ------------------------------------------- 8-bit activation checkpoints
 * x [T,H] (MOE_F32 | MOE_BF16) <-> codes int8 [T,H], scales uint8 [T,H/32]:
 * per block of 32 values of a row one power-of-two step 2^(scale - 127), and
 *   code = rint(x / step), half to even;  value = code * step,
 * the step being the smallest power of two with every |code| <= 127 (never
 * below 2^-126, never above 2^121: there codes are held at +-127).  So
 * |value - x| <= step / 2 <= max|x of the block| / 127, x / step is exact, and
 * every value is exact in bf16 as well as in fp32.  A block that holds a NaN
 * or an infinity gets scale 255 and codes 0: all its values are NaN.
 * H a positive multiple of 32; T = 0 is a no-op. */
int moe_act_pack8(const void *x, int x_dtype, int T, int H, int8_t *codes, uint8_t *scales, moe_stream_t s);
int moe_act_unpack8(const int8_t *codes, const uint8_t *scales, int T, int H, void *x, int x_dtype,
                    moe_stream_t s);

/* ------------------------------------------------ balance loss and counts
 * Over the N tokens that token_mask (device uint8 [T], 0 = padding; NULL = all
 * count) leaves, with p[t,:] = softmax(logits[t,:]) over all E experts and
 * lse[t] = log sum_e exp(logits[t,e]):
 *   counts[e] = number of (t, j) with topk_ids[t,j] = e;  counts[E] = N
 *   f[e]      = counts[e] / (N k)
 *   balance   = E * sum_e f[e] * mean_t p[t,e]
 *   z         = mean_t lse[t]^2
 *   loss[4]   = { balance_coef * balance + z_coef * z, balance, z, N }
 * counts device int32 [E+1] out, loss device fp32 [4] out.  The logits of
 * masked tokens are not read.  N = 0 gives zeros.  A token whose logits are
 * all -inf adds nothing to the sums (its ids are counted).  A NaN or +inf
 * logit of a counted token sets MOE_DEVERR_NONFINITE and makes the losses NaN;
 * an id outside [0,E) sets MOE_DEVERR_BAD_EXPERT and is not counted.
 * Sums over a warp's tokens are held in fp32 (of lse^2 in fp64), over warps in
 * fp64.
 * 1 <= E <= 32768, 1 <= k <= min(E,32), T * k <= 2^30.  ws: at least
 * moe_balance_ws_size(T,E) bytes.  token_mask needs no alignment. */
size_t moe_balance_ws_size(int T, int E);
int moe_balance_loss(const float *logits, const int32_t *topk_ids, const uint8_t *token_mask, int T, int E, int k,
                     float balance_coef, float z_coef, int32_t *counts, float *loss, void *ws, size_t ws_bytes,
                     moe_stream_t s);

/* Gradient of the router's logits: of loss[0] above times *d_loss, plus, when
 * d_topk_w is given, of the gates (the softmax over the k selected logits):
 *   d_logits[t,e] = d_loss * p[t,e] * ( balance_coef * E / N * (f[e] - sum_i f[i] p[t,i])
 *                                       + z_coef * 2 * lse[t] / N )
 *                 + sum over j with topk_ids[t,j] = e of
 *                     topk_w[t,j] * (d_topk_w[t,j] - sum_i topk_w[t,i] d_topk_w[t,i])
 * counts int32 [E+1] as moe_balance_loss left them (held constant; sums over
 * several devices' tokens may be put in their place, f and N follow), or NULL:
 * no loss term.  d_loss device fp32 scalar (4-byte aligned) or NULL for 1.
 * topk_w/d_topk_w device fp32 [T,k], or both NULL: no gate term.  logits may
 * be NULL without a loss term, topk_ids without a gate term.  d_logits
 * device [T,E] out (not logits itself), dl_dtype MOE_F32 | MOE_BF16 (rounded once).  Rows of
 * masked tokens are written as zeros and none of their inputs is read. */
int moe_route_backward(const float *logits, const int32_t *topk_ids, const float *topk_w, const float *d_topk_w,
                       const uint8_t *token_mask, const int32_t *counts, const float *d_loss, int T, int E, int k,
                       float balance_coef, float z_coef, void *d_logits, int dl_dtype, moe_stream_t s);

/* ------------------------------------------ backward pass of the experts
 * For y[t] = sum_j topk_w[t,j] FFN_e(x_t) (+ FFN_shared(x_t)), e = topk_ids[t,j]
 * (moe_expert_ffn_* then moe_combine), given dy = dL/dy:
 *   g = Wg x, u = Wu x, s = 1 / (1 + exp(-g)), a = g s, q = Wd^T dy
 *   d_topk_w[t,j] = sum_i q_i a_i u_i
 *   dx[t] = sum_j topk_w[t,j] (Wg^T (q u (s + a (1 - s))) + Wu^T (q a))  (+ the shared expert's)
 * g and u are recomputed from x, so that x is all the forward pass keeps.
 *  expert_blobs, expert_offsets, active, perm_src, perm_dst, topk_w: as in the
 *           forward pass.  Every expert of the step has to be in `active`: a
 *           row whose expert is not, or has no blob, adds nothing to dx and
 *           gets d_topk_w 0 (a NULL blob also sets MOE_DEVERR_NULL_BLOB).
 *           So does a row whose expert's entry is wrong (MOE_DEVERR_BAD_EXPERT,
 *           _BAD_ROW, _MISALIGNED).  Where the lists name more rows than T k by
 *           so much that GEMM mode cannot hold them, MOE_DEVERR_BAD_ROW is set
 *           and no row is computed, the shared expert's neither: dx and
 *           d_topk_w are zero.  After MOE_DEVERR_TIMEOUT the call's outputs are
 *           not to be used.
 *  x        device [T,H]: MOE_F32 | MOE_BF16 (x_scales NULL), or MOE_Q8, the
 *           codes and x_scales of moe_act_pack8.
 *  dy       device [T,H], MOE_F32 | MOE_BF16.
 *  dx       device [T,H] out, MOE_F32 | MOE_BF16 (rounded once).
 *  d_topk_w device [T,k] fp32 out.
 *  mode     MOE_MODE_GEMV: CUDA cores, fp32 throughout, any T.
 *           MOE_MODE_GEMM: tcgen05 tensor cores.  Operands are rounded to
 *           fp16 (half a step: 2^-11 of the value): the weights, each token's x
 *           and dy, and, between the two products, the gradients of g and u.
 *           x and dy are divided by a power of two of the token's own, the
 *           gradients of g and u by one of the token's and one of the expert's
 *           (all undone in fp32), so that neither x's, dy's nor the weights'
 *           scale matters and nothing leaves fp16's range, but for a weight
 *           that is itself outside: a step above 65504 / 2^(bits-1), infinite
 *           or NaN sets MOE_DEVERR_NONFINITE, and the rows of its expert may
 *           not be finite.  fp32 accumulation.  Blobs in device memory.
 *           MOE_MODE_AUTO: GEMV up to 4 tokens, else GEMM, with its fp16
 *           operands; a caller that wants fp32 throughout asks for GEMV.
 *  Shapes as for moe_expert_ffn_*: H a multiple of 128 up to 8192, I up to 4096.
 *  ws: at least moe_expert_ffn_backward_ws_size(...) bytes. */
size_t moe_expert_ffn_backward_ws_size(int bits, int T, int k, int H, int I, int E, int mode);
int moe_expert_ffn_backward(int bits, const void *const *expert_blobs, const int32_t *expert_offsets,
                            const int32_t *active, const int32_t *perm_src, const int32_t *perm_dst,
                            const float *topk_w, const void *x, int x_dtype, const uint8_t *x_scales,
                            const void *dy, int dy_dtype, int T, int k, int H, int I, int E,
                            const void *shared_blob, void *dx, int dx_dtype, float *d_topk_w, int mode, void *ws,
                            size_t ws_bytes, moe_stream_t s);

/* ----------------------------------------- backward pass of the router
 * For logits = x W^T + bias:
 *   dx       = dx_in + d_logits W      (dx_in device [T,H] fp32 or NULL)
 *   d_w      = d_logits^T x            [E,H], in w_dtype (rounded once)
 *   d_bias   = sum_t d_logits[t,:]     [E] fp32
 * d_logits [T,E], x [T,H] and w [E,H] are MOE_F32 | MOE_BF16; dx is dx_dtype.
 * Any of dx, d_w, d_bias may be NULL (not computed); dx may be dx_in itself
 * when dx_dtype is MOE_F32.  With the three dtypes MOE_BF16 and E a multiple
 * of 8 the products run on the tensor cores (fp32 accumulation; d_w's sum over
 * tokens in up to one part per SM, added in order), else in fp32 on CUDA cores.
 * T = 0 writes zeros to d_w and d_bias.
 * T <= 2^30, H a positive multiple of 8, 1 <= E <= 32768.  ws: at least
 * moe_router_backward_ws_size(...) bytes (may be 0: then ws may be NULL). */
size_t moe_router_backward_ws_size(int T, int H, int E, int dl_dtype, int x_dtype, int w_dtype);
int moe_router_backward(const void *d_logits, int dl_dtype, const void *x, int x_dtype, const void *w_router,
                        int w_dtype, const float *dx_in, int T, int H, int E, void *dx, int dx_dtype, void *d_w,
                        float *d_bias, void *ws, size_t ws_bytes, moe_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H_ */
