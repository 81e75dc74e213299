/*
 * forge_layer.h -- the operators of a training step around the fused weight step (forge.h) that
 * a layer with expert (mixture-of-experts) weights needs: the RMS norm before the products, the
 * products grouped by expert, and the optimizer's step of every parameter the fused step does
 * not take.
 *
 * The conventions of forge.h hold here: row-major contiguous tensors (ld == cols) on 16-byte
 * aligned device pointers of the current device, caller-owned buffers, no device allocation,
 * arguments checked before anything is enqueued on `stream`, statuses and forge_last_error().
 */
#ifndef FORGE_LAYER_H
#define FORGE_LAYER_H

#include <stdint.h>

#include "forge.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Where the scale of an FP8_E4M3 output comes from. */
#define FORGE_SCALE_ROW 0    /* written: y->scale receives one fp32 scale per row */
#define FORGE_SCALE_TENSOR 1 /* given: y->scale holds one fp32 scale for the tensor */

/*
 * forge_rmsnorm -- RMS norm of x (+ residual), optionally to fp8.  For every row t:
 *     h    = x + residual, rounded to the dtype of x (nearest even); h = x without a residual
 *     rstd = 1 / sqrt(mean(h^2) + eps)            (of the rounded h, in fp32)
 *     y    = (h * rstd) * gain
 *   x, residual, h   [T, D], all F32 or all BF16.  residual and h are both given or both NULL;
 *                    h may be x or residual itself (in place), else it overlaps no input.
 *   gain             [1, D], F32 or BF16.
 *   y                [T, D] F32, BF16 (nearest even) or FP8_E4M3.  FP8: y holds
 *                    rne_e4m3(clamp(y / scale, -448, 448)), the quotients rounded to fp32, with
 *                      FORGE_SCALE_ROW     scale = max(amax_t |y| / 448, 2^-126), written to
 *                                          y->scale[t] (T fp32);
 *                      FORGE_SCALE_TENSOR  scale = y->scale[0], read (> 0): the per-tensor form
 *                                          forge_wgrad_step takes as X.
 *                    scale_mode is ignored for other dtypes.  A row holding NaN or an infinity
 *                    gives NaN (scale and codes) wherever the formula does.
 *   rstd             T fp32 or NULL.
 *   amax             one fp32 or NULL: raised to max |y| over the tensor where that is larger
 *                    (the caller sets it to 0 first; NaN sticks), for the next tensor scale.
 * D is any length from 1 to 2^31 - 1, T below 2^31, every tensor below 2^48 bytes; rows of D <= 16384 take
 * one pass over memory, fastest where D % 8 == 0.
 */
forge_status forge_rmsnorm(const forge_tensor* x, const forge_tensor* residual, const forge_tensor* gain, float eps,
                           forge_tensor* h, forge_tensor* y, int32_t scale_mode, float* rstd, float* amax,
                           void* stream);

/*
 * forge_rmsnorm_backward -- gradients of forge_rmsnorm (unquantised y) for one upstream dy:
 *     a  = dy * gain,  u = h * rstd
 *     dx = rstd * (a - u * mean(a * u)) + dh     (the gradient of x and of residual)
 *     dgain[d] = sum_t dy * u
 *   dy, dh, h, dx    [T, D], all F32 or all BF16; dh (the gradient arriving on h itself) may be
 *                    NULL.  dx may be dy or dh itself, else it overlaps no input.  h may instead be
 *                    codes (FP8_B128 or I8_B128 of forge_ffn.h, scale [T, ceil(D / 128)]): the
 *                    formula then takes what they stand for, beside the rstd of the h that was.
 *   rstd             T fp32, as forge_rmsnorm wrote it.
 *   dgain            [1, D] F32, overwritten; NULL where it is not needed.  The sum over rows has
 *                    a fixed order: the same inputs give the same bits.
 *   workspace        forge_rmsnorm_backward_workspace_bytes(T, D) bytes, 16-byte aligned,
 *                    overlapping no tensor; unused (may be NULL) without dgain.
 */
forge_status forge_rmsnorm_backward(const forge_tensor* dy, const forge_tensor* dh, const forge_tensor* h,
                                    const forge_tensor* gain, const float* rstd, forge_tensor* dx,
                                    forge_tensor* dgain, void* workspace, int64_t workspace_bytes, void* stream);
int64_t forge_rmsnorm_backward_workspace_bytes(int64_t T, int64_t D); /* -1 for negative or huge sizes */

/*
 * Products grouped by expert.  The rows of X [T, K] and dY [T, N] are sorted by expert: group e
 * is rows ends[e - 1] .. ends[e] - 1 (from 0 for e = 0), `ends` being n_groups int32 on the
 * device, ascending, in [0, T].  Groups may be empty; rows past the last end belong to no expert.
 * The library cannot check device data: an end outside [0, T] is taken as the nearer bound and an
 * end below its predecessor as an empty group.  W [n_groups * N, K] holds the experts' weights
 * [N, K] one after another.  N and K are multiples of 128, N K < 2^31, 1 <= n_groups <= 4096.
 *
 * forge_grouped_gemm   Y[t] = X[t] W_e^T for every row t of group e; rows of no group get zeros.
 *                      X, W BF16; or both FP8_E4M3 with X->scale T and W->scale n_groups * N fp32
 *                      (one per row).  fp32 accumulation; Y [T, N] BF16, nearest even.  The fp8
 *                      matrix instructions cut the products of each eight consecutive contraction
 *                      elements at 2^-13 of the largest one's power of two before they add them.
 * forge_grouped_dgrad  dX[t] = dY[t] W_e, likewise (all BF16).
 * forge_grouped_wgrad  dW_e = dY_e^T X_e for every group, fp32 [n_groups * N, K] (zeros for an
 *                      empty group); X, dY BF16, each below 4 GiB with 128 rows more (here and in
 *                      the step).
 * forge_grouped_wgrad_step  the same gradient, applied to every expert's weight by rule `opt` in
 *                      the product's epilogue as forge_wgrad_step does (an empty group takes the
 *                      step with a zero gradient); W BF16 with n_groups N K < 2^32, m, v as there.
 *                      Stochastic rounding counts elements over the whole of W.
 */
forge_status forge_grouped_gemm(const forge_tensor* X, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                forge_tensor* Y, void* stream);
forge_status forge_grouped_dgrad(const forge_tensor* dY, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                 forge_tensor* dX, void* stream);
forge_status forge_grouped_wgrad(const forge_tensor* X, const forge_tensor* dY, const int32_t* ends, int32_t n_groups,
                                 forge_tensor* dW, void* stream);
forge_status forge_grouped_wgrad_step(const forge_tensor* X, const forge_tensor* dY, const int32_t* ends,
                                      int32_t n_groups, forge_tensor* W, forge_tensor* m, forge_tensor* v,
                                      const forge_hyper* hyper, int32_t opt, int64_t step, uint64_t seed,
                                      const forge_step_opts* opts, void* stream);

/*
 * One optimizer step over many tensors in one launch (parameters with a materialised gradient:
 * norm gains, biases, embeddings, weights of any size).  A tensor is n consecutive elements,
 * 0 <= n <= 2^32 - 8192, all together fewer than 2^36; the moments of all tensors of a table are fp32, or all 8-bit in blocks of 64 of
 * the same map (I8_B64 / U8_B64 or I8DYN_B64 / U8DYN_B64, ceil(n / 64) fp32 scales each; the
 * last block may be short).
 */
typedef struct forge_multi_tensor {
  void* W;            /* F32 or BF16 */
  const void* g;      /* gradient, F32 or BF16 */
  void* m;            /* NULL for a moment the rule does not keep */
  void* v;
  float* m_scale;     /* NULL for fp32 moments */
  float* v_scale;
  int64_t n;
  uint64_t seed;      /* stochastic-rounding key of this tensor (BF16 weights) */
  int32_t w_dtype, g_dtype;
  int32_t group;      /* which entry of the step's hyper-parameters it takes, 0 .. 7 */
  int32_t reserved;   /* 0 */
} forge_multi_tensor;

/* What the host knows of a packed table. */
typedef struct forge_multi_info {
  int64_t bytes;      /* of the table */
  int64_t chunks;     /* workgroups of a step */
  int32_t tensors, groups; /* groups: one more than the largest group used */
  int32_t opt, m_dtype, v_dtype; /* dtypes: -1 for a moment the rule does not keep */
  int32_t reserved;
} forge_multi_info;

/* Bytes of the table of these tensors (-1: a negative or too large n, or too many elements). */
int64_t forge_multi_table_bytes(const forge_multi_tensor* tensors, int32_t n_tensors);
/*
 * forge_multi_pack -- host only: checks the tensors for rule `opt` and moments of dtype m_dtype /
 * v_dtype (ignored for a moment the rule does not keep) and writes the table to the host buffer
 * `table`; the caller copies it to the device (16-byte aligned) and keeps it, with the tensors,
 * for the steps.  It is to be packed anew when a pointer changes.  Pointers must be 16-byte
 * aligned (scales 4); nothing written may overlap anything else of the table.
 */
forge_status forge_multi_pack(const forge_multi_tensor* tensors, int32_t n_tensors, int32_t opt, int32_t m_dtype,
                              int32_t v_dtype, void* table, int64_t table_bytes, forge_multi_info* info);
/*
 * forge_multi_step -- one step of the packed tensors.  table: the packed table on the device.
 * hypers: n_hypers >= info->groups (at most 8) hyper-parameter sets, one for each group.
 * grad_scale: one fp32 on the device that every gradient is multiplied by (a clipping or
 * unscaling factor), or NULL.  Rounding of BF16 weights and its random bits: as
 * forge_optimizer_step (sr_enable of opts; w_preround_out must be NULL).
 */
forge_status forge_multi_step(const forge_multi_info* info, const void* table, const forge_hyper* hypers,
                              int32_t n_hypers, int64_t step, const float* grad_scale, const forge_step_opts* opts,
                              void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FORGE_LAYER_H */
