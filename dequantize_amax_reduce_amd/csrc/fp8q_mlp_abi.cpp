// fp8q_mlp_abi.cpp -- the C ABI declared in include/fp8q_mlp.h.
//
// As in fp8q_abi.cpp, every entry point validates its arguments on the host
// first (no HIP call, no side effect) and only then enqueues kernels.
#include "fp8q_mlp.h"

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "fp8q_ffn_check.h"
#include "fp8q_mlp_launch.h"

namespace {

// n zeros of an element type
void zeros(void* p, int64_t n, int dt, hipStream_t st) {
    if (!p || n == 0) return;
    if (dt == FP8Q_F32) fp8q::launch_fill_f32((float*)p, n, 0.0f, st);
    else fp8q::launch_zero16(p, n, st);
}

fp8q_status_t layernorm(const fp8q::LayerNorm& a, void* stream) {
    const bool plain = a.to == fp8q::kToPlain, group = a.to == fp8q::kToGroup;
    if (!valid_dtype(a.dt) || (!plain && !valid_fmt(a.fmt)) || (a.wdt != a.dt && a.wdt != FP8Q_F32)) return FP8Q_EDTYPE;
    if (a.rows < 0 || a.cols < 0) return FP8Q_EINVAL;
    if (group && a.cols % 128 != 0) return FP8Q_ESHAPE;
    if (a.rows > kMaxNormRows || a.cols > kMaxNormCols) return FP8Q_EINVAL;
    const int64_t n = a.rows * a.cols, es = esize(a.dt), we = esize(a.wdt);
    const int64_t sc = plain ? 0 : group ? a.rows * (a.cols / 128) : a.rows;
    if (a.rows == 0) return FP8Q_OK;
    if ((n > 0 && (!a.x || !a.w || !a.y)) || (sc > 0 && !a.sinv)) return FP8Q_EINVAL;
    if (!aligned(a.x, es) || !aligned(a.res, es) || !aligned(a.h, es) || !aligned(a.w, we) || !aligned(a.b, we) ||
        (plain && !aligned(a.y, es)) || !aligned(a.sinv, 4) || !aligned(a.mean, 4) || !aligned(a.rstd, 4))
        return FP8Q_EALIGN;
    const Buf out[] = {{a.y, plain ? n * es : n}, {a.h, n * es}, {a.sinv, 4 * sc}, {a.mean, a.mean ? 4 * a.rows : 0},
                       {a.rstd, a.rstd ? 4 * a.rows : 0}, {a.w, a.cols * we}, {a.b, a.cols * we}};
    if (bad_overlap(out, 7, 5)) return FP8Q_EINVAL;
    // h, and y in x's type, may be x or the residual itself; otherwise the outputs meet nothing
    for (const void* in : {a.x, a.res})
        for (int i = 0; i < 5; ++i)
            if (overlap(out[i], {in, n * es}) && !(out[i].p == in && (i == 1 || (i == 0 && plain)))) return FP8Q_EINVAL;
    if (a.cols == 0) {
        if (a.to != fp8q::kToRow) return FP8Q_OK;
        fp8q::launch_fill_f32(a.sinv, a.rows, 1.0f, S(stream));
        return launched();
    }
    fp8q::launch_layernorm(a, S(stream));
    return launched();
}

fp8q_status_t linear_act(fp8q::MmAct& e, int64_t M, int64_t N, int64_t K, void* stream) {
    fp8q::MmFwd& f = e.f;
    if (!valid_fmt(f.xfmt) || !valid_fmt(f.wfmt) || !valid_unary(f.act) || (e.bias && !valid_dtype(e.bdt)) ||
        (f.z && !valid_dtype(f.zdt)))
        return FP8Q_EDTYPE;
    fp8q_status_t st = check_sizes(M, N, K, kMaxFwdRows);
    if (st != FP8Q_OK) return st;
    if (!grid_ok(M, N)) return FP8Q_EINVAL;
    if (M == 0 || N == 0) return FP8Q_OK;
    if (f.q ? !f.sinv : !f.y) return FP8Q_EINVAL;
    for (const Codes& c : {Codes{f.x, f.xs, M, M}, Codes{f.w0, f.ws0, N, blocks(N)}}) {
        st = check_codes(c, K);
        if (st != FP8Q_OK) return st;
    }
    const int64_t n = M * N, ye = esize(f.ydt);
    if (!aligned(f.y, ye) || !aligned(e.res, ye) || (f.z && !aligned(f.z, esize(f.zdt))) || !aligned(f.sinv, 4) ||
        (e.bias && !aligned(e.bias, esize(e.bdt))))
        return FP8Q_EALIGN;
    const int64_t wsb = fp8q::mm_act_workspace(M, N, K, f.q != nullptr);
    st = check_ws(f.ws, wsb);
    if (st != FP8Q_OK) return st;
    const int64_t KB = K / 128;
    // y may be the residual
    const Buf b[] = {{f.y, n * ye}, {f.z, f.z ? n * esize(f.zdt) : 0}, {f.q, n}, {f.sinv, 4 * M * (N / 128)}, {f.ws, wsb},
                     {e.res, e.res == f.y ? 0 : n * ye}, {e.bias, e.bias ? N * esize(e.bdt) : 0}, {f.x, M * K},
                     {f.xs, 4 * M * KB}, {f.w0, N * K}, {f.ws0, 4 * blocks(N) * KB}};
    if (bad_overlap(b, 11, 5)) return FP8Q_EINVAL;
    f.M = M;
    f.N = (int)N;
    f.K = (int)K;
    fp8q::launch_mm_act(e, S(stream));
    return launched();
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------

fp8q_status_t fp8q_layernorm(const void* x, fp8q_dtype_t xdtype, const void* residual, const void* weight,
                             const void* bias, fp8q_dtype_t wdtype, int64_t rows, int64_t cols, float eps, void* y,
                             void* h, float* mean, float* rstd, void* stream) {
    return layernorm({x, xdtype, residual, weight, bias, wdtype, rows, cols, eps, fp8q::kToPlain, 0, y, nullptr, h, mean,
                      rstd}, stream);
}

fp8q_status_t fp8q_layernorm_cast_group128(const void* x, fp8q_dtype_t xdtype, const void* residual,
                                           const void* weight, const void* bias, fp8q_dtype_t wdtype, int64_t rows,
                                           int64_t cols, float eps, fp8q_fmt_t fmt, uint8_t* q, float* scale_inv,
                                           void* h, float* mean, float* rstd, void* stream) {
    return layernorm({x, xdtype, residual, weight, bias, wdtype, rows, cols, eps, fp8q::kToGroup, fmt, q, scale_inv, h,
                      mean, rstd}, stream);
}

fp8q_status_t fp8q_layernorm_cast_per_channel(const void* x, fp8q_dtype_t xdtype, const void* residual,
                                              const void* weight, const void* bias, fp8q_dtype_t wdtype, int64_t rows,
                                              int64_t cols, float eps, fp8q_fmt_t fmt, uint8_t* q, float* scale_inv,
                                              void* h, float* mean, float* rstd, void* stream) {
    return layernorm({x, xdtype, residual, weight, bias, wdtype, rows, cols, eps, fp8q::kToRow, fmt, q, scale_inv, h,
                      mean, rstd}, stream);
}

size_t fp8q_layernorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows > kMaxNormRows || cols > kMaxNormCols) return 0;
    return (size_t)(fp8q::layernorm_bwd_parts(rows) * cols * 8);
}

fp8q_status_t fp8q_layernorm_backward(const void* dy, const void* h, fp8q_dtype_t dtype, const void* weight,
                                      fp8q_dtype_t wdtype, const float* mean, const float* rstd, const void* dh,
                                      int64_t rows, int64_t cols, void* dx, void* dweight, void* dbias,
                                      void* workspace, void* stream) {
    if (!valid_dtype(dtype) || (wdtype != dtype && wdtype != FP8Q_F32)) return FP8Q_EDTYPE;
    if (rows < 0 || cols < 0 || rows > kMaxNormRows || cols > kMaxNormCols) return FP8Q_EINVAL;
    const int64_t n = rows * cols, es = esize(dtype), we = esize(wdtype);
    if (cols == 0) return FP8Q_OK;
    if (n > 0 && (!dy || !h || !weight || !mean || !rstd || !dx)) return FP8Q_EINVAL;
    if (!aligned(dy, es) || !aligned(h, es) || !aligned(dh, es) || !aligned(dx, es) || !aligned(weight, we) ||
        !aligned(dweight, we) || !aligned(dbias, we) || !aligned(mean, 4) || !aligned(rstd, 4))
        return FP8Q_EALIGN;
    const int64_t wsb = dweight || dbias ? (int64_t)fp8q_layernorm_backward_workspace_bytes(rows, cols) : 0;
    const fp8q_status_t st = check_ws(workspace, wsb);
    if (st != FP8Q_OK) return st;
    // dx may be dy or dh, but then that tensor still may not meet another output
    const Buf b[] = {{dx, n * es}, {dweight, cols * we}, {dbias, cols * we}, {workspace, wsb},
                     {dy, dx == dy ? 0 : n * es}, {dh, dx == dh ? 0 : n * es}, {h, n * es}, {weight, cols * we},
                     {mean, 4 * rows}, {rstd, 4 * rows}};
    if (bad_overlap(b, 10, 4)) return FP8Q_EINVAL;
    if (rows == 0) {
        zeros(dweight, cols, wdtype, S(stream));
        zeros(dbias, cols, wdtype, S(stream));
        return dweight || dbias ? launched() : FP8Q_OK;
    }
    fp8q::launch_layernorm_bwd({dy, h, dtype, weight, wdtype, mean, rstd, dh, rows, cols, dx, dweight, dbias,
                                (float*)workspace}, S(stream));
    return launched();
}

// ---------------------------------------------------------------------------
// projection with an epilogue
// ---------------------------------------------------------------------------

size_t fp8q_linear_act_workspace_bytes(int64_t M, int64_t N, int64_t K, int cast) {
    if (!sizes_ok(M, N, K, kMaxFwdRows)) return 0;
    return (size_t)fp8q::mm_act_workspace(M, N, K, cast != 0);
}

fp8q_status_t fp8q_linear_act(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w,
                              fp8q_fmt_t wfmt, const float* w_scale_inv, int64_t M, int64_t N, int64_t K,
                              const void* bias, fp8q_dtype_t bdtype, fp8q_act_t act, const void* residual, void* y,
                              fp8q_dtype_t ydtype, void* z, fp8q_dtype_t zdtype, void* workspace, void* stream) {
    if (!valid_dtype(ydtype)) return FP8Q_EDTYPE;
    fp8q::MmAct e{};
    fp8q::MmFwd& f = e.f;
    f.x = x; f.xs = x_scale_inv; f.w0 = w; f.ws0 = w_scale_inv; f.xfmt = xfmt; f.wfmt = wfmt; f.act = act;
    f.y = y; f.ydt = ydtype; f.z = z; f.zdt = zdtype; f.ws = workspace;
    e.bias = bias; e.bdt = bdtype; e.res = residual;
    return linear_act(e, M, N, K, stream);
}

fp8q_status_t fp8q_linear_act_cast(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w,
                                   fp8q_fmt_t wfmt, const float* w_scale_inv, int64_t M, int64_t N, int64_t K,
                                   const void* bias, fp8q_dtype_t bdtype, fp8q_act_t act, fp8q_fmt_t fmt, uint8_t* q,
                                   float* scale_inv, void* z, fp8q_dtype_t zdtype, void* workspace, void* stream) {
    if (!valid_fmt(fmt)) return FP8Q_EDTYPE;
    if (M < 0 || N < 0) return FP8Q_EINVAL;
    if (N % 128 != 0) return FP8Q_ESHAPE;
    if (M > 0 && N > 0 && !q) return FP8Q_EINVAL;
    fp8q::MmAct e{};
    fp8q::MmFwd& f = e.f;
    f.x = x; f.xs = x_scale_inv; f.w0 = w; f.ws0 = w_scale_inv; f.xfmt = xfmt; f.wfmt = wfmt; f.act = act;
    f.q = q; f.qfmt = fmt; f.sinv = scale_inv; f.z = z; f.zdt = zdtype; f.ws = workspace;
    e.bias = bias; e.bdt = bdtype;
    return linear_act(e, M, N, K, stream);
}

size_t fp8q_linear_act_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!sizes_ok(M, N, K, kMaxRows)) return 0;
    return (size_t)fp8q::mm_act_bwd_workspace(M, N, K);
}

fp8q_status_t fp8q_linear_act_backward(const void* dy, const void* z, fp8q_dtype_t dtype, const uint8_t* x,
                                       fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w, fp8q_fmt_t wfmt,
                                       const float* w_scale_inv, int64_t M, int64_t N, int64_t K, fp8q_act_t act,
                                       void* dx, void* dw, void* dbias, fp8q_dtype_t dwdtype, void* workspace,
                                       void* stream) {
    if (!half_dtype(dtype) || !valid_fmt(xfmt) || !valid_fmt(wfmt) || !valid_unary(act) ||
        (dwdtype != dtype && dwdtype != FP8Q_F32))
        return FP8Q_EDTYPE;
    fp8q_status_t st = check_sizes(M, N, K, kMaxRows);
    if (st != FP8Q_OK) return st;
    if (!grid_ok(M, K) || !grid_ok(2 * N + 64, K)) return FP8Q_EINVAL;
    // the layout pass: 64 x 64 tiles of dy, 64 x 128 of the codes, 256 threads each
    const int64_t mt = M / 64 + 2, nt = N / 64 + 2;         // both are padded to 64 or 128
    if (mt * nt + (K / 128) * (mt + nt) >= int64_t(1) << 24) return FP8Q_EINVAL;
    const int64_t n = M * N;
    const void* zin = act == FP8Q_IDENTITY ? nullptr : z;
    if (n > 0 && (!dy || (act != FP8Q_IDENTITY && !z))) return FP8Q_EINVAL;
    const bool products = K > 0 && (dx || dw);
    if (n > 0 && products) {
        for (const Codes& c : {Codes{x, x_scale_inv, M, M}, Codes{w, w_scale_inv, N, 0}}) {
            st = check_codes(c, K);
            if (st != FP8Q_OK) return st;
        }
    }
    const int64_t we = esize(dwdtype), KB = K / 128;
    if (!aligned(dy, 2) || !aligned(zin, 2) || !aligned(dx, 2) || !aligned(dw, we) || !aligned(dbias, we)) return FP8Q_EALIGN;
    if (!products && !dbias) return FP8Q_OK;
    const int64_t wsb = fp8q::mm_act_bwd_workspace(M, N, K);
    st = check_ws(workspace, wsb);
    if (st != FP8Q_OK) return st;
    const Buf b[] = {{dx, M * K * 2}, {dw, N * K * we}, {dbias, N * we}, {workspace, wsb}, {dy, n * 2}, {zin, n * 2},
                     {x, M * K}, {x_scale_inv, 4 * M * KB}, {w, N * K}, {w_scale_inv, 4 * blocks(N) * KB}};
    if (bad_overlap(b, 10, 4)) return FP8Q_EINVAL;
    // empty outputs: dx without rows, dw and dbias without columns
    const bool any = (dx && M > 0 && K > 0) || (dw && N > 0 && K > 0) || (dbias && N > 0);
    if (!any) return FP8Q_OK;
    fp8q::MmActBwd e{};
    fp8q::MmBwd& f = e.f;
    f.dy = dy; f.z = zin; f.dt = dtype; f.x = x; f.xs = x_scale_inv; f.w0 = w; f.ws0 = w_scale_inv;
    f.M = M; f.N = (int)N; f.K = (int)K; f.xfmt = xfmt; f.wfmt = wfmt; f.act = act;
    f.dx = dx; f.dw0 = dw; f.dwdt = dwdtype; f.ws = workspace; e.db = dbias;
    fp8q::launch_mm_act_bwd(e, S(stream));
    return launched();
}

}  // extern "C"
