/*
 * fp8q_mlp.h -- C ABI of the operators of blocks with layer norm and biased
 * projections: what fp8q_ffn.h offers for blocks with RMS norm and gated
 * projections, for AMD Instinct MI355X (gfx950).
 *
 * The conventions of fp8q.h and fp8q_ffn.h hold (device pointers, dense
 * row-major tensors, fp8 activations and weights and their scales as there,
 * asynchronous on `stream`, arguments validated on the host before any HIP
 * call, no allocation, no state kept, the same limits and workspaces), and the
 * calling thread's current device is the one that holds the tensors.
 *
 * Numerics are those of fp8q_ffn.h: a projection of more than 64 rows whose outputs
 * are all 16-bit uses the fp8 instruction, which adds a step's products within
 * about 16 bits of the largest; a binary32 y or z, a cast, and up to 64 rows have
 * binary32 sums.  A row's result does not depend on what the other rows hold; its
 * last bits may depend on how many there are, which choose the tiles and the splits
 * of a contraction.
 */
#ifndef FP8Q_MLP_H
#define FP8Q_MLP_H

#include "fp8q_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual addition, layer norm, and its result in x's type or cast to fp8:
 *   h = x (+ residual, in binary32);  mean[r] = mean_c h[r, c];
 *   rstd[r] = 1 / sqrt(mean_c (h[r, c] - mean[r])^2 + eps);
 *   y = ((h - mean[r]) * rstd[r]) * weight[c] (+ bias[c]), in binary32, from the
 *   sum before its rounding to xdtype;
 *   fp8q_layernorm:                  y rounded once to xdtype;
 *   fp8q_layernorm_cast_group128:    q, scale_inv = the cast of y per 128
 *     columns, by fp8q_cast_per_group128's rule (scale_inv [rows, cols/128];
 *     cols % 128 != 0 -> FP8Q_ESHAPE);
 *   fp8q_layernorm_cast_per_channel: per row, by fp8q_cast_per_channel's rule
 *     (scale_inv [rows]).
 * x, residual, h, y: [rows, cols] of xdtype.  residual may be NULL (h = x).
 * h may be NULL (not written) and may be x or residual itself (in place); y may
 * be x or residual itself where it is not h.
 * weight, bias: [cols] of wdtype, which is xdtype or FP8Q_F32 (else
 * FP8Q_EDTYPE); bias may be NULL.  mean, rstd: [rows] floats, or NULL.
 * The mean is taken twice, the second time of the differences from the first,
 * so that rows far from zero lose nothing but h's own rounding, and a constant
 * row has y = bias.  (Of rows too long for registers, past 32768 16-bit or 16384
 * binary32 columns, and of rows under 16 bytes, it is a binary64 sum's.)  Sums are
 * binary32: a row whose sum passes 3.4e38 may get NaN, and one whose differences
 * pass 1.8e19 gets rstd = 0, as an infinite variance gives it.  Short rows are
 * summed in another order where there are more than 256 of them.
 * rows == 0 is a no-op; cols == 0 is a no-op except that the per-channel form
 * writes scale_inv[r] = 1 (mean and rstd are not written).
 */
fp8q_status_t fp8q_layernorm(const void* x, fp8q_dtype_t xdtype, const void* residual, const void* weight,
                             const void* bias, fp8q_dtype_t wdtype, int64_t rows, int64_t cols, float eps, void* y,
                             void* h, float* mean, float* rstd, void* stream);
fp8q_status_t fp8q_layernorm_cast_group128(const void* x, fp8q_dtype_t xdtype, const void* residual,
                                           const void* weight, const void* bias, fp8q_dtype_t wdtype, int64_t rows,
                                           int64_t cols, float eps, fp8q_fmt_t fmt, uint8_t* q, float* scale_inv,
                                           void* h, float* mean, float* rstd, void* stream);
fp8q_status_t fp8q_layernorm_cast_per_channel(const void* x, fp8q_dtype_t xdtype, const void* residual,
                                              const void* weight, const void* bias, fp8q_dtype_t wdtype, int64_t rows,
                                              int64_t cols, float eps, fp8q_fmt_t fmt, uint8_t* q, float* scale_inv,
                                              void* h, float* mean, float* rstd, void* stream);

/*
 * Backward of the layer norm (the cast passes gradients through).  dy [rows,
 * cols] is the gradient of y; h, mean and rstd are the forward's; dh (or NULL)
 * is the gradient that reaches h along the residual path:
 *   n = (h - mean) * rstd;  dn = dy * weight;
 *   dx = (dn - mean_c(dn) - n * mean_c(dn * n)) * rstd + dh;
 *   dweight[c] = sum_r dy * n;  dbias[c] = sum_r dy.
 * dx (the gradient of x and of the residual alike) may be dy or dh itself.
 * dy, h, dh, dx: dtype; weight, dweight, dbias: wdtype (dtype or FP8Q_F32).
 * dweight and dbias may be NULL each.  rows == 0 writes zeros to them.
 * workspace: fp8q_layernorm_backward_workspace_bytes(rows, cols) bytes, needed
 * only with dweight or dbias.
 */
size_t fp8q_layernorm_backward_workspace_bytes(int64_t rows, int64_t cols);
fp8q_status_t fp8q_layernorm_backward(const void* dy, const void* h, fp8q_dtype_t dtype, const void* weight,
                                      fp8q_dtype_t wdtype, const float* mean, const float* rstd, const void* dh,
                                      int64_t rows, int64_t cols, void* dx, void* dweight, void* dbias,
                                      void* workspace, void* stream);

/*
 * One projection with a bias, an activation and a residual in its epilogue:
 *   z = X W^T (+ bias[n]) in binary32  [M, N];
 *   fp8q_linear_act:      y = act(z) (+ residual), rounded once to ydtype;
 *   fp8q_linear_act_cast: q, scale_inv = the per-128-group cast of act(z) (from
 *     binary32, fp8q_cast_per_group128's rule); N % 128 != 0 -> FP8Q_ESHAPE.
 * act: any fp8q_act_t; act(-infinity) is 0 but of FP8Q_IDENTITY.  bias: [N] of bdtype, any element type, or NULL.
 * residual: [M, N] of ydtype, or NULL; y may be the residual itself (in place).
 * z (or NULL): [M, N] of zdtype, each value rounded once: what the backward
 * pass reads.  K == 0 gives z = bias; M == 0 or N == 0 is a no-op.
 * workspace: fp8q_linear_act_workspace_bytes(M, N, K, cast) bytes, cast = 1 for
 *   fp8q_linear_act_cast.
 */
size_t fp8q_linear_act_workspace_bytes(int64_t M, int64_t N, int64_t K, int cast);
fp8q_status_t fp8q_linear_act(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w,
                              fp8q_fmt_t wfmt, const float* w_scale_inv, int64_t M, int64_t N, int64_t K,
                              const void* bias, fp8q_dtype_t bdtype, fp8q_act_t act, const void* residual, void* y,
                              fp8q_dtype_t ydtype, void* z, fp8q_dtype_t zdtype, void* workspace, void* stream);
fp8q_status_t fp8q_linear_act_cast(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w,
                                   fp8q_fmt_t wfmt, const float* w_scale_inv, int64_t M, int64_t N, int64_t K,
                                   const void* bias, fp8q_dtype_t bdtype, fp8q_act_t act, fp8q_fmt_t fmt, uint8_t* q,
                                   float* scale_inv, void* z, fp8q_dtype_t zdtype, void* workspace, void* stream);

/*
 * Its backward, from dy [M, N] (the gradient of y or of the cast's values; the
 * residual's gradient is dy itself) and the forward's z [M, N]:
 *   dz = dy * act'(z) in binary32;  dx [M, K] = dz W;  dw [N, K] = dz^T X;
 *   dbias[n] = sum_m dz, in binary32 from the unrounded dz.
 * act' of FP8Q_RELU is 0 from 0 down; at -infinity and infinity a slope is 0 and
 * 1.  With FP8Q_IDENTITY dz = dy and z is not
 * read (it may be NULL).  dy and z are bf16 or f16 (FP8Q_F32 -> FP8Q_EDTYPE); dx
 * has their type, dw and dbias dwdtype: that type or FP8Q_F32.  dx, dw and dbias
 * may each be NULL (not computed).  The operands of the two products, their
 * precision and the limits are those of fp8q_linear_backward, with an activation
 * those of fp8q_gated_linear_backward.  M == 0 writes dw = 0 and dbias = 0, N == 0
 * dx = 0.
 * workspace: fp8q_linear_act_backward_workspace_bytes(M, N, K) bytes.
 */
size_t fp8q_linear_act_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);
fp8q_status_t fp8q_linear_act_backward(const void* dy, const void* z, fp8q_dtype_t dtype, const uint8_t* x,
                                       fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w, fp8q_fmt_t wfmt,
                                       const float* w_scale_inv, int64_t M, int64_t N, int64_t K, fp8q_act_t act,
                                       void* dx, void* dw, void* dbias, fp8q_dtype_t dwdtype, void* workspace,
                                       void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP8Q_MLP_H */
