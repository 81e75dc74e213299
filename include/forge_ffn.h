/*
 * forge_ffn.h -- the operators of a gated feed-forward block beside those of forge_layer.h: both
 * projections with the activation in one product and its backward pass, activation checkpoints in 8
 * bits with the backward passes that read them, and matrix products of fp8 codes with a scale for
 * each block of 128.
 *
 * The conventions of forge.h hold here: row-major contiguous tensors (ld == cols) on 16-byte
 * aligned device pointers of the current device, caller-owned buffers, no device allocation,
 * arguments checked before anything is enqueued on `stream`, statuses and forge_last_error().
 * Groups (`ends`, `n_groups`) are those of forge_layer.h; a dense layer is one group of all rows.
 */
#ifndef FORGE_FFN_H
#define FORGE_FFN_H

#include <stdint.h>

#include "forge.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Codes of blocks of 128 columns (dtypes FORGE_FP8_B128 and FORGE_I8_B128).  A tensor [T, D] has
 * ceil(D / 128) fp32 scales a row (`scale`, [T, ceil(D / 128)], the last block may be short), and
 * an element stands for code * scale:
 *     scale = max(amax / most, 2^-126),  code = rne(x * (1 / scale)),
 * with most = 448 for e4m3 codes and 127 for int8 ones; the quotients and the product are rounded
 * to fp32.  A block that holds NaN or an infinity gets a NaN scale and zero codes: all of it reads
 * back as NaN.
 *
 * forge_block_quantize    q = codes of x.  x [T, D] F32 or BF16; q FP8_B128 or I8_B128.
 * forge_block_dequantize  y = code * scale, rounded to F32 or BF16 (nearest even).
 *   D below 2^31, T * ceil(D / 128) below 2^47; fastest where D % 8 == 0.
 */
forge_status forge_block_quantize(const forge_tensor* x, forge_tensor* q, void* stream);
forge_status forge_block_dequantize(const forge_tensor* q, forge_tensor* y, void* stream);

/*
 * forge_block_quantize_weight -- e4m3 codes of n_groups weights W [n_groups * N, K] (F32 or BF16) in
 * squares of 128 x 128, by the same rule: q [n_groups * N, K] FP8_B128 with `scale`
 * [n_groups, N / 128, K / 128].  qt (or NULL): the transposed weights [n_groups * K, N] with `scale`
 * [n_groups, K / 128, N / 128], the same codes, which the input gradient takes as its weight.
 * N and K are multiples of 128.
 */
forge_status forge_block_quantize_weight(const forge_tensor* W, int32_t n_groups, forge_tensor* q, forge_tensor* qt,
                                         void* stream);

/*
 * forge_grouped_block_gemm -- for the rows t of group e, with X [T, K] codes by rows and W
 * [n_groups * N, K] codes by squares (both FP8_B128, scales as above):
 *     Y[t, n] = sum over blocks b of (sx[t, b] sw_e[n / 128, b]) * sum over k in b of X[t, k] W_e[n, k]
 * Y [T, N] BF16, nearest even; rows of no group get zeros.  A block's sum is fp32, formed as
 * forge_grouped_gemm's fp8 products are (forge_layer.h), and so is the sum over blocks.  The product of
 * two scales is rounded to fp32: it has to stay in fp32's range, and below 2^-126 loses bits.
 * With qt as W it gives the input gradient of codes dY.  Sizes as forge_grouped_gemm.
 */
forge_status forge_grouped_block_gemm(const forge_tensor* X, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                      forge_tensor* Y, void* stream);

/* Activations of a gated product. */
#define FORGE_ACT_SILU 0      /* g / (1 + exp(-g)) */
#define FORGE_ACT_GELU 1      /* g * (1 + erf(g / sqrt 2)) / 2 */
#define FORGE_ACT_GELU_TANH 2 /* g * (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */
#define FORGE_ACT_RELU 3      /* max(g, 0), slope 0 at 0 */

/*
 * forge_grouped_gated -- for the rows t of group e, W [n_groups * 2 N, K] holding every group's gate
 * rows [N, K] and then its up rows [N, K]:
 *     g = X[t] Wg^T,  u = X[t] Wu^T,  H[t] = act(g) * u
 *   X, W     BF16; fp32 accumulation, and the activation takes the fp32 sums.
 *   H        [T, N] BF16, nearest even; rows of no group get zeros.
 *   gate_up  [T, 2 N] or NULL: g in columns 0 .. N - 1 and u in N .. 2 N - 1, as the backward pass
 *            takes them: BF16 (nearest even), or FP8_B128 / I8_B128 codes of the fp32 sums
 *            (scale [T, 2 N / 128]).
 * N and K are multiples of 128, 2 N and K at most 2^20, 2 N K < 2^31.
 */
forge_status forge_grouped_gated(const forge_tensor* X, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                 int32_t act, forge_tensor* H, forge_tensor* gate_up, void* stream);

/*
 * Backward pass of H = act(g) * u from the gradient dH of H:
 *     dg = dH * u * act'(g),  du = dH * act(g),  H = act(g) * u
 * with g and u what gate_up stands for (it is not rounded further).  dgate_up [T, 2 N] has dg beside du,
 * as the gradient of the stacked product: forge_grouped_dgrad of it with W gives dX, and
 * forge_grouped_wgrad or _step of X with it the weight's.  H (or NULL) is the input that the weight
 * gradient of the down projection takes.  The activations and their slopes are fp32 operations, whose
 * exponentials carry a rounding of their exponent x (g, g^2 / 2 for GELU): |x| 2^-23 of their value.  Exponentials and
 * act(g) / g below 2^-126 count as zero: act(g) of g below -87 (SiLU), -13.2 (GELU) or -10 (GELU_TANH).
 *
 * forge_gated_backward  dH [T, N], dgate_up [T, 2 N] and H [T, N] all F32 or all BF16; gate_up of the
 *   same dtype, or codes with scale [T, 2, ceil(N / 128)]: blocks begin anew at u.  Any N from 1 to
 *   2^30.  H may be dH itself, and dgate_up gate_up itself (in both), else nothing written overlaps an input.
 * forge_grouped_gated_dgrad  the same with dH = dY W_e for the rows of group e, in fp32, never stored: dY
 *   [T, K] the gradient of the down projection's output, W [n_groups * K, N] its weights, BF16; gate_up BF16
 *   or codes; dgate_up, H BF16.  Rows of no group get zeros.  N and K as forge_grouped_dgrad's.
 */
forge_status forge_gated_backward(const forge_tensor* dH, const forge_tensor* gate_up, int32_t act,
                                  forge_tensor* dgate_up, forge_tensor* H, void* stream);
forge_status forge_grouped_gated_dgrad(const forge_tensor* dY, const forge_tensor* W, const int32_t* ends,
                                       int32_t n_groups, const forge_tensor* gate_up, int32_t act,
                                       forge_tensor* dgate_up, forge_tensor* H, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FORGE_FFN_H */
