/*
 * fp8q_ffn.h -- C ABI of the feed-forward operators on fp8 operands: the
 * layers that produce fp8q.h's codes and scales and the matrix products that
 * consume them, with their backward passes, for AMD Instinct MI355X (gfx950).
 *
 * The conventions of fp8q.h hold (device pointers, dense row-major tensors,
 * asynchronous on `stream`, arguments validated on the host before any HIP
 * call, no allocation, no state kept, FP8Q_OK or the first error found), and:
 *  - An fp8 activation X [M, K] is what fp8q_cast_per_group128 writes: codes
 *    and x_scale_inv [M, K/128]; X[m, k] = fp32(x[m, k]) * x_scale_inv[m, k/128].
 *  - An fp8 weight W [N, K] has one scale per 128x128 block, as
 *    fp8q_weight_dequant_block128 reads it: w_scale_inv [ceil(N/128), K/128],
 *    W[n, k] = fp32(w[n, k]) * w_scale_inv[n/128, k/128].
 *  - K % 128 != 0 -> FP8Q_ESHAPE.  The codes of X and W are read 16 bytes at a
 *    time: a base address that is not 16-byte aligned -> FP8Q_EALIGN (rows are
 *    whole multiples of 128 bytes).  Other pointers need only their element's
 *    alignment; 16-byte aligned ones are faster.
 *  - K, N and F are at most 2^21, M at most 2^31 (4194240 in the backward
 *    passes), a product has fewer than 2^23 tiles of 64 x 128 outputs, and a
 *    backward pass fewer than 2^24 tiles of 64 x 64 operand elements
 *    (FP8Q_EINVAL beyond).  Norms take up to 2^31 - 1 rows of up to 2^30.
 *  - A workspace is scratch for one call: its contents need no initialisation
 *    and hold nothing the caller reads.  It is 256-byte aligned, owned by the
 *    caller and not shared with a call that may run at the same time.  A NULL
 *    workspace is accepted where the size function gives 0.  A backward pass
 *    lays its operands out there in f16, on every call: about 4 M C + 2 K (C + M)
 *    bytes with C = N, and half as much again with C = 2 F for a gated pair (1.8
 *    GB for M = 4096, K = 7168, F = 18432), and binary32 partial sums where a
 *    contraction is split.
 *  - Outputs do not overlap inputs or one another unless an entry point says
 *    so.
 *
 * Numerics
 *  - fp8 x fp8 products are exact.  They are summed over each 128-long block
 *    of K, and the block's sum times its two scales is added to a binary32
 *    accumulator (one FMA).  Outputs are rounded once.  The sums within a block
 *    are binary32 wherever an output shows it (a binary32 y, h or z, or an fp8
 *    cast with its scales); where every output is bf16 or f16 and M > 64, the
 *    fp8 matrix instruction sums the block, with about 16 bits kept below the
 *    block's largest product (up to 4e-5 of the sum's rms measured).
 *  - Every sum has a fixed order: the same call gives the same bits.  The order,
 *    the splits of K and the kind of sum are chosen from M, N and K, so a row's
 *    last bits may differ between calls of different M (another kernel from 17
 *    rows on, the fp8 instruction from 65 on).
 *  - NaN and infinities follow the formulas (0 * inf is NaN).
 *  - Backward products take their operands in f16, each rounded once, and sum
 *    in binary32.  The largest scale of each row of X, and of each block row of
 *    W, goes to the gradient's operand (a projection's as a power of two, which
 *    leaves a 16-bit dy exact); then a power of two brings the largest finite
 *    value of every row (for dx) or column (for dw) of the gradient's operand, and
 *    of every 128 columns of K of X's and W's, under 2^15.  They are taken off the
 *    sums.  So a row of dx does not depend on the other rows of the gradient, a
 *    row of X or a block row of W that meets no gradient changes nothing whatever
 *    its scale, and gradients of any magnitude need no scaling: values down to
 *    2^-28 of the largest of their row, column or 128 columns keep 11 bits.  A
 *    gated pair's f16 gradients take the rounding's rest of dz too, to 3 bits.
 *    In root mean square f16 gradients are about 3e-4 off (2.1e-4 is their own
 *    rounding), bf16 ones 1.7e-3 (1.66e-3).
 *  - The gradient of a cast is the identity: gradients are those of the
 *    formulas at the values the codes stand for.
 */
#ifndef FP8Q_FFN_H
#define FP8Q_FFN_H

#include "fp8q.h"

#ifdef __cplusplus
extern "C" {
#endif

/* activation of the gate: x / (1 + exp(-x)); x * Phi(x) with the error
 * function; and its tanh form x/2 * (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
typedef enum { FP8Q_SILU = 0, FP8Q_GELU = 1, FP8Q_GELU_TANH = 2 } fp8q_act_t;

/*
 * Residual addition, root-mean-square norm, cast to fp8:
 *   h = x (+ residual, in binary32);  rstd[r] = 1 / sqrt(mean_c h[r, c]^2 + eps);
 *   y = (h * rstd[r]) * weight[c], in binary32, from the sum before its
 *   rounding to xdtype;  q, scale_inv = the cast of y:
 *   fp8q_rmsnorm_cast_group128:   per 128 columns, by fp8q_cast_per_group128's
 *     rule (scale_inv [rows, cols/128]; cols % 128 != 0 -> FP8Q_ESHAPE);
 *   fp8q_rmsnorm_cast_per_channel: per row, by fp8q_cast_per_channel's rule
 *     (scale_inv [rows]).
 * x, residual, h: [rows, cols] of xdtype.  residual may be NULL (h = x).
 * h may be NULL (not written) and may be x or residual itself (in place).
 * weight: [cols] of wdtype, which is xdtype or FP8Q_F32 (else FP8Q_EDTYPE).
 * The sum of squares is binary32: a row with values past 1.8e19 gets rstd = 0,
 * as an infinite mean gives it.
 * rstd: [rows] floats, or NULL.  rows == 0 is a no-op; cols == 0 is a no-op
 * except that the per-channel form writes scale_inv[r] = 1 and, for both,
 * rstd is not written.
 */
fp8q_status_t fp8q_rmsnorm_cast_group128(const void* x, fp8q_dtype_t xdtype, const void* residual, const void* weight,
                                         fp8q_dtype_t wdtype, int64_t rows, int64_t cols, float eps, fp8q_fmt_t fmt,
                                         uint8_t* q, float* scale_inv, void* h, float* rstd, void* stream);
fp8q_status_t fp8q_rmsnorm_cast_per_channel(const void* x, fp8q_dtype_t xdtype, const void* residual,
                                            const void* weight, fp8q_dtype_t wdtype, int64_t rows, int64_t cols,
                                            float eps, fp8q_fmt_t fmt, uint8_t* q, float* scale_inv, void* h,
                                            float* rstd, void* stream);

/*
 * Backward of the norm (the cast passes gradients through).  dy [rows, cols]
 * is the gradient of y; h and rstd are the forward's; dh (or NULL) is the
 * gradient that reaches h along the residual path:
 *   n = h * rstd;  dn = dy * weight;
 *   dx = (dn - n * mean_c(dn * n)) * rstd + dh;   dweight[c] = sum_r dy * n.
 * dx (the gradient of x and of the residual alike) may be dy or dh itself.
 * dy, h, dh, dx: dtype; weight, dweight: wdtype (dtype or FP8Q_F32).
 * dweight may be NULL.  rows == 0 writes dweight = 0 (dweight not NULL).
 * workspace: fp8q_rmsnorm_backward_workspace_bytes(rows, cols) bytes, needed
 * only with dweight.
 */
size_t fp8q_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols);
fp8q_status_t fp8q_rmsnorm_backward(const void* dy, const void* h, fp8q_dtype_t dtype, const void* weight,
                                    fp8q_dtype_t wdtype, const float* rstd, const void* dh, int64_t rows, int64_t cols,
                                    void* dx, void* dweight, void* workspace, void* stream);

/*
 * One projection: y [M, N] = X W^T, rounded once to ydtype.
 * K == 0 writes zeros; M == 0 or N == 0 is a no-op.
 * workspace: fp8q_linear_workspace_bytes(M, N, K) bytes.
 */
size_t fp8q_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);
fp8q_status_t fp8q_linear(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w,
                          fp8q_fmt_t wfmt, const float* w_scale_inv, int64_t M, int64_t N, int64_t K, void* y,
                          fp8q_dtype_t ydtype, void* workspace, void* stream);

/*
 * Its backward: dx [M, K] = dy W, dw [N, K] = dy^T X.  dy is bf16 or f16
 * (FP8Q_F32 -> FP8Q_EDTYPE); dx has dy's type; dw has dwdtype: dy's type or
 * FP8Q_F32.  Either of dx and dw may be NULL (not computed).
 * M == 0 writes dw = 0; N == 0 writes dx = 0.
 * workspace: fp8q_linear_backward_workspace_bytes(M, N, K) bytes.
 */
size_t fp8q_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);
fp8q_status_t fp8q_linear_backward(const void* dy, fp8q_dtype_t dtype, const uint8_t* x, fp8q_fmt_t xfmt,
                                   const float* x_scale_inv, const uint8_t* w, fp8q_fmt_t wfmt,
                                   const float* w_scale_inv, int64_t M, int64_t N, int64_t K, void* dx, void* dw,
                                   fp8q_dtype_t dwdtype, void* workspace, void* stream);

/*
 * Gate and up projections, the activation and the product:
 *   g = X Wg^T, u = X Wu^T (binary32);  p = act(g) * u  [M, F].
 * fp8q_gated_linear: h = p rounded once to hdtype.
 * fp8q_gated_linear_cast: q, scale_inv = the per-128-group cast of p (from
 *   binary32, fp8q_cast_per_group128's rule); F % 128 != 0 -> FP8Q_ESHAPE.
 * z (or NULL): [M, 2 F] of zdtype, g in columns [0, F) and u in [F, 2 F), each
 *   rounded once: what the backward pass reads.
 * w_gate, w_up: [F, K] codes of wfmt (the two halves of a merged weight, or
 *   two tensors).  K == 0 gives g = u = 0; M == 0 or F == 0 is a no-op.
 * workspace: fp8q_gated_linear_workspace_bytes(M, F, K, cast) bytes, cast = 1
 *   for fp8q_gated_linear_cast.
 */
size_t fp8q_gated_linear_workspace_bytes(int64_t M, int64_t F, int64_t K, int cast);
fp8q_status_t fp8q_gated_linear(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w_gate,
                                const float* w_gate_scale_inv, const uint8_t* w_up, const float* w_up_scale_inv,
                                fp8q_fmt_t wfmt, int64_t M, int64_t F, int64_t K, fp8q_act_t act, void* h,
                                fp8q_dtype_t hdtype, void* z, fp8q_dtype_t zdtype, void* workspace, void* stream);
fp8q_status_t fp8q_gated_linear_cast(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv,
                                     const uint8_t* w_gate, const float* w_gate_scale_inv, const uint8_t* w_up,
                                     const float* w_up_scale_inv, fp8q_fmt_t wfmt, int64_t M, int64_t F, int64_t K,
                                     fp8q_act_t act, fp8q_fmt_t fmt, uint8_t* q, float* scale_inv, void* z,
                                     fp8q_dtype_t zdtype, void* workspace, void* stream);

/*
 * Its backward, from dp [M, F] (the gradient of p) and the forward's z:
 *   dg = dp * u * act'(g), du = dp * act(g)  (binary32, then an operand);
 *   dx [M, K] = dg Wg + du Wu;  dw_gate [F, K] = dg^T X;  dw_up = du^T X.
 * dp and z have dtype, bf16 or f16; dx too; dw_gate and dw_up have dwdtype
 * (dtype or FP8Q_F32).  dx may be NULL, and dw_gate and dw_up may both be.
 * M == 0 writes zero weight gradients; F == 0 writes dx = 0.
 * workspace: fp8q_gated_linear_backward_workspace_bytes(M, F, K) bytes.
 */
size_t fp8q_gated_linear_backward_workspace_bytes(int64_t M, int64_t F, int64_t K);
fp8q_status_t fp8q_gated_linear_backward(const void* dp, const void* z, fp8q_dtype_t dtype, const uint8_t* x,
                                         fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w_gate,
                                         const float* w_gate_scale_inv, const uint8_t* w_up,
                                         const float* w_up_scale_inv, fp8q_fmt_t wfmt, int64_t M, int64_t F, int64_t K,
                                         fp8q_act_t act, void* dx, void* dw_gate, void* dw_up, fp8q_dtype_t dwdtype,
                                         void* workspace, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP8Q_FFN_H */
