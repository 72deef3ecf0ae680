/*
 * tee_train.h -- the operators a training step of the encoder adds to the
 * forward pass (same library as tee.h): the LayerNorm, the scaled token lookup
 * and the softmax cross entropy over the vocabulary, each forward and backward.
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

#ifdef __cplusplus
}
#endif
#endif /* TEE_TRAIN_H */
