/*
 * tee_train.h -- the operators a training step of the encoder adds to the
 * forward pass (same library as tee.h): the LayerNorm, the scaled token lookup,
 * the softmax cross entropy over the vocabulary, rotary positions, attention and
 * the gated half of the feed-forward block, each forward and backward, and the
 * clipping of all gradients by their common norm.
 *
 * As in tee_ops.h every call runs on caller-provided DEVICE buffers,
 * asynchronously on `stream` (a cudaStream_t, NULL = legacy default stream), on
 * the device of `ctx`, which also supplies the status word and the error
 * message; the current device of the caller is left as it was.  The context's
 * weights are not used (they need not be loaded): a training program owns its
 * parameters, so tables, gains and gradients are arguments.  No call allocates
 * device memory, synchronises or keeps anything between calls, so all of them
 * can be captured into a CUDA graph; scratch memory is the caller's (d_ws,
 * ws_bytes, at least what the operator's *_workspace function returns; its
 * contents need no initialisation and mean nothing afterwards).  Calls that may
 * overlap on the GPU need a workspace each.
 *
 * Buffers are row-major and contiguous.  Element types are given as TEE_F32
 * (float) or TEE_BF16 (bfloat16, uint16 bit patterns); any other value is
 * TEE_EINVAL.  Buffers are 16-byte aligned (int32 and statistics arrays and the
 * per-position floats: 4-byte aligned, statistics 8); a NULL or misaligned
 * buffer or a workspace that is too small returns TEE_EINVAL before anything is
 * launched.  Outputs must not overlap inputs except where stated.  Results do
 * not depend on the order in which thread blocks run: the same inputs give the
 * same bits.
 *
 * Arithmetic: inputs are widened to fp32, sums and statistics are fp32 (the
 * products of the vocabulary loss take bf16 operands into fp32 accumulators),
 * outputs are rounded once to their type.
 */
#ifndef TEE_TRAIN_H
#define TEE_TRAIN_H

#include <stddef.h>
#include <stdint.h>
#include "tee.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- LayerNorm (bias-free, as tee_op_layernorm) ---------------------------
 *   mean_t = sum_h x[t,h] / H,  rstd_t = 1 / sqrt(sum_h (x[t,h] - mean_t)^2 / H + eps)
 *   y[t,h] = (x[t,h] - mean_t) rstd_t gamma[h]
 * 1 <= H <= TEE_LN_MAX_HIDDEN; T >= 0 rows. */
#define TEE_LN_MAX_HIDDEN 8192

/* y y_type[T*H], stats float[T*2] ({mean, rstd} per row, for the backward pass;
 * NULL if not wanted) from x x_type[T*H] and gamma float[H].  d_y may be d_x
 * where the types are the same. */
int tee_op_layernorm_forward(tee_ctx* ctx, const void* d_x, int x_type, const float* d_gamma, void* d_y, int y_type,
                             float* d_stats, int T, int H, float eps, void* stream);

/* With xhat = (x - mean) rstd and u = dy gamma:
 *   dx[t,h]   = rstd_t (u[t,h] - sum_h u[t,h] / H - xhat[t,h] sum_h u[t,h] xhat[t,h] / H) + dres[t,h]
 *   dgamma[h] = sum_t dy[t,h] xhat[t,h]
 * dy y_type[T*H]; x, dres (the gradient that reaches x past the norm, as on a
 * residual branch; NULL for none) and dx x_type[T*H]; stats as the forward pass
 * wrote them.  d_dx may be d_dres, or d_x or d_dy where the types are the same.
 * With T == 0 dgamma is set to zero. */
int tee_op_layernorm_backward(tee_ctx* ctx, const void* d_dy, int y_type, const void* d_x, int x_type,
                              const float* d_gamma, const float* d_stats, const void* d_dres, void* d_dx,
                              float* d_dgamma, int T, int H, void* d_ws, size_t ws_bytes, void* stream);
long long tee_layernorm_backward_workspace(int T, int H);

/* ---- token lookup with scaling ---------------------------------------------
 *   y[t] = scale E[id[t]],   E table_type[V*H], ids int32[T], y y_type[T*H]
 * An id outside [0, V) gives a zero row and sets the context's device status
 * (tee_device_status), as in tee_op_embed.  1 <= H <= 65536, V >= 1. */
int tee_op_embed_forward(tee_ctx* ctx, const void* d_table, int table_type, const int32_t* d_ids, void* d_y, int y_type,
                         int T, int V, int H, float scale, void* stream);

/* The table's gradient:  dE[v] (+)= scale sum_{t: id[t] = v} dy[t], the tokens
 * of a row added in a fixed order (the tokens are sorted by id, stably).
 * dy y_type[T*H], dE table_type[V*H].  accumulate 0: every row of dE is written,
 * rows without a token with zeros; 1: rows with tokens are added to (in fp32,
 * rounded once) and the others left alone, as for a table that also has the
 * gradient of the vocabulary loss.  A token whose id is outside [0, V) adds
 * nothing and sets the device status. */
int tee_op_embed_backward(tee_ctx* ctx, const void* d_dy, int y_type, const int32_t* d_ids, void* d_dtable,
                          int table_type, int T, int V, int H, float scale, int accumulate, void* d_ws,
                          size_t ws_bytes, void* stream);
long long tee_embed_backward_workspace(int T, int V, int H);

/* ---- softmax cross entropy over the vocabulary -------------------------------
 * Masked-token prediction with the token table as the output weight.  For the
 * counted positions i (those whose target is not ignore_id):
 *   logit[i,v] = x[i] . w[v],   lse[i] = log sum_v exp logit[i,v],
 *   loss[i] = lse[i] - logit[i, target[i]]
 * and loss[i] = lse[i] = 0 for the others, which cost no products and whose
 * states are not looked at.  The logits are not kept, not even for one position:
 * both passes work through them tile by tile.  A target that is neither
 * ignore_id nor in [0, V) is treated as ignored and sets the device status.
 *   x bf16[N*H], w bf16[V*H], targets int32[N], loss and lse float[N];
 *   H a multiple of 8 in [8, TEE_VOCAB_MAX_HIDDEN]; 0 <= N <= 2^24,
 *   1 <= V <= 2^24, and ceil(N / 256) ceil(V / 256) <= 2^30.
 * Logits are fp32; those past 2^127 in magnitude count as infinite.  A wait inside
 * the products that does not end gives TEE_ETIMEOUT from the next
 * tee_device_status, as in the tensor-core projections. */
#define TEE_VOCAB_MAX_HIDDEN 8192
int tee_op_vocab_loss_forward(tee_ctx* ctx, const void* d_x, const void* d_w, const int32_t* d_targets, float* d_loss,
                              float* d_lse, int N, int V, int H, int ignore_id, void* d_ws, size_t ws_bytes,
                              void* stream);
long long tee_vocab_loss_forward_workspace(int N, int V, int H);

/* With g[i] the gradient that reaches loss[i] (1 / their number for the mean over
 * the counted positions) and D[i,v] = g[i] (exp(logit[i,v] - lse[i]) - [v == target[i]]):
 *   dx[i] = sum_v D[i,v] w[v]   (0 for positions that are not counted),
 *   dw[v] = sum_i D[i,v] x[i]
 * gloss float[N], lse as the forward pass wrote it, dx bf16[N*H], dw bf16[V*H];
 * d_dx or d_dw may be NULL where that gradient is not wanted (not both).  D is
 * rounded to bf16, as the other operands of these products are (its rows first
 * divided by the largest |g|), with two exceptions: up to 128 counted positions it
 * keeps a second bf16 half, and in dx the target's entry counts whole.  The rounding
 * of the outputs costs 1.7e-3 of their norm; with D's, dw is 1.9e-3 to 2.3e-3 off.
 * exp(logit - lse) - 1 at the target is as exact as lse in fp32 is: its sign and size
 * hold down to about 2^-24 |lse|.  More than 65536 positions are taken in equal
 * parts, whose dw is added in fp32.
 * Every row of dw is written, zeros where nothing reaches it, also with N == 0; a
 * table that is also looked up gets the lookup's gradient added by
 * tee_op_embed_backward with accumulate 1, which rounds a row with tokens again. */
int tee_op_vocab_loss_backward(tee_ctx* ctx, const void* d_x, const void* d_w, const int32_t* d_targets,
                               const float* d_lse, const float* d_gloss, void* d_dx, void* d_dw, int N, int V, int H,
                               int ignore_id, void* d_ws, size_t ws_bytes, void* stream);
long long tee_vocab_loss_backward_workspace(int N, int V, int H);

/* ---- rotary positions --------------------------------------------------------
 * On packed rows of n_heads queries, n_heads keys and n_heads values of 64 columns
 * each (qkv, as tee_op_attention takes them).  For every query and key head,
 * j < 32, with the angle a = pos[t] base^(-j / 32):
 *   y[j] = x[j] cos a - x[j + 32] sin a,  y[j + 32] = x[j + 32] cos a + x[j] sin a
 * and the values are copied.  The backward pass turns by the negated angle.
 * x and y type[T * 192 n_heads]; pos int32[T], as tee_op_positions gives them; d_y
 * may be d_x (the values then stay).  1 <= n_heads <= TEE_ATTN_MAX_HEADS, base > 0.
 * Angles are taken in 64 bits, to within 1e-7 of a turn. */
#define TEE_ATTN_MAX_HEADS 512
int tee_op_rope_forward(tee_ctx* ctx, const void* d_x, int type, const int32_t* d_pos, void* d_y, int T, int n_heads,
                        float base, void* stream);
int tee_op_rope_backward(tee_ctx* ctx, const void* d_dy, int type, const int32_t* d_pos, void* d_dx, int T, int n_heads,
                         float base, void* stream);

/* ---- attention ------------------------------------------------------------------
 * Bidirectional attention inside each text of a packed batch, as tee_op_attention,
 * for a step that is going to be differentiated.  Row i sees the rows j of its text,
 * with window >= 0 those with |i - j| <= window.  Per head of 64 columns:
 *   s[i,j] = q[i] . k[j] / 8,  lse[i] = log sum_j exp s[i,j],
 *   o[i] = sum_j exp(s[i,j] - lse[i]) v[j]
 * qkv bf16[T * 192 n_heads] (rotated, where positions are); cu int32[n_texts + 1] on
 * the DEVICE: cu[0] = 0, cu not decreasing, cu[n_texts] <= T, at most
 * TEE_ATTN_MAX_TEXT_TOKENS tokens to a text.  Other offsets set the device status
 * and leave the outputs as they were.  Texts may be empty.  Rows behind the last
 * text are not written, and what they hold has no effect, were it NaN, but all T rows
 * of every buffer have to be there: tiles reach into them.  No text's results depend
 * on another's values: they are the same bits whatever finite ones those are.  Next to
 * values that are not finite a row may be computed another way, to the same error bound.
 * Values that are not finite give infinities or NaN in the rows and columns that they
 * reach by the formulas, and in no others.
 * o bf16[T * 64 n_heads], lse float[n_heads * T], head by head.
 * 0 <= T <= 2^24, 0 <= n_texts <= 2^20.  The host sees neither cu nor the texts'
 * lengths, so one captured graph serves batches of other texts.
 * The products take bf16 operands into fp32 accumulators: the probabilities are
 * rounded to bf16 for the product with v (not for lse), and the gradients' factors
 * likewise. */
#define TEE_ATTN_MAX_TEXT_TOKENS 131072
int tee_op_attention_forward(tee_ctx* ctx, const void* d_qkv, const int32_t* d_cu, void* d_o, float* d_lse, int T,
                             int n_texts, int n_heads, int window, void* d_ws, size_t ws_bytes, void* stream);
long long tee_attention_forward_workspace(int T, int n_texts, int n_heads);

/* With p[i,j] = exp(s[i,j] - lse[i]), delta[i] = do[i] . o[i] and
 * ds[i,j] = p[i,j] (do[i] . v[j] - delta[i]):
 *   dq[i] = sum_j ds[i,j] k[j] / 8,  dk[j] = sum_i ds[i,j] q[i] / 8,  dv[j] = sum_i p[i,j] do[i]
 * The probabilities are computed again.  o and lse as the forward pass wrote them,
 * do bf16[T * 64 n_heads]; dqkv bf16[T * 192 n_heads] in the layout of qkv, of whose
 * queries and keys tee_op_rope_backward makes the gradients before their rotation. */
int tee_op_attention_backward(tee_ctx* ctx, const void* d_qkv, const int32_t* d_cu, const void* d_o, const float* d_lse,
                              const void* d_do, void* d_dqkv, int T, int n_texts, int n_heads, int window, void* d_ws,
                              size_t ws_bytes, void* stream);
long long tee_attention_backward_workspace(int T, int n_texts, int n_heads);

/* ---- the gated half of the feed-forward block ---------------------------------------
 * As tee_op_ffn_in: both projections, the activation and the product, in one launch.
 *   a = x wa^T, g = x wg^T,  z = GELU(a) g      (GELU(a) = a Phi(a))
 * x bf16[T*H]; wi bf16[2I*H], the rows of wa and then those of wg; z bf16[T*I].
 * H a multiple of 8 in [8, TEE_GEGLU_MAX_HIDDEN], I one in [8, TEE_GEGLU_MAX_WIDTH],
 * 0 <= T <= 2^24. */
#define TEE_GEGLU_MAX_HIDDEN 8192
#define TEE_GEGLU_MAX_WIDTH 32768
int tee_op_geglu_forward(tee_ctx* ctx, const void* d_x, const void* d_wi, void* d_z, int T, int H, int I, void* stream);

/* Nothing but x is kept from the forward pass; a and g are computed again.
 *   da = dz g GELU'(a), dg = dz GELU(a)   (rounded to bf16 for the products below)
 *   dx = da wa + dg wg,   dwi = [da^T x; dg^T x]
 * dz bf16[T*I], dx bf16[T*H], dwi bf16[2I*H]; d_dx or d_dwi may be NULL where that
 * gradient is not wanted (not both).  With T == 0 dwi is set to zero.  More than 65536
 * rows are taken in equal parts, whose dwi is added in fp32. */
int tee_op_geglu_backward(tee_ctx* ctx, const void* d_x, const void* d_wi, const void* d_dz, void* d_dx, void* d_dwi, int T,
                          int H, int I, void* d_ws, size_t ws_bytes, void* stream);
long long tee_geglu_backward_workspace(int T, int H, int I);

/* ---- clipping by the common norm ------------------------------------------------------
 * Of n_tensors gradients, h_grads[i] with h_counts[i] elements of type h_types[i]:
 *   norm = sqrt(sum of all squares),  factor = min(1, max_norm / norm),  out = factor g
 * factor is 1 where the norm is zero, infinite or not a number: such gradients are
 * passed on as they are, and norm tells.  d_norm float[2] = {norm, factor}.
 * The four lists are HOST arrays, read before the call returns; the tensors are on the
 * device, contiguous, aligned to their elements (16 bytes: faster).  h_outs[i] may be
 * h_grads[i] (where factor is 1 it is then not written); no output may overlap another
 * or another tensor's gradient otherwise.  h_outs NULL: all in place.  Counts may be 0.
 * max_norm >= 0, infinity for the norm alone.  Squares are summed without overflow
 * or underflow whatever the magnitudes.  0 <= n_tensors <= 65536.  TEE_ENOMEM where the
 * host has no memory to compare the tensors' places. */
int tee_op_clip_gradients(tee_ctx* ctx, const void* const* h_grads, const int32_t* h_types, const int64_t* h_counts,
                          void* const* h_outs, int n_tensors, float max_norm, float* d_norm, void* d_ws,
                          size_t ws_bytes, void* stream);
long long tee_clip_gradients_workspace(int n_tensors);

#ifdef __cplusplus
}
#endif
#endif /* TEE_TRAIN_H */
