// fp8q_ffn_abi.cpp -- the C ABI declared in include/fp8q_ffn.h.
//
// As in fp8q_abi.cpp, every entry point validates its arguments on the host
// first (no HIP call, no side effect) and only then enqueues kernels.
#include "fp8q_ffn.h"

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "fp8q_ffn_launch.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 21;    // K, N, F
constexpr int64_t kMaxRows = 65535 * 64;         // M of a backward pass
constexpr int64_t kMaxNormRows = INT32_MAX, kMaxNormCols = int64_t(1) << 30;
constexpr int64_t kMaxTiles = (int64_t(1) << 23) - 1;   // workgroups of 512 threads: 2^32 threads a grid

bool valid_dtype(int dt) { return dt == FP8Q_F32 || dt == FP8Q_BF16 || dt == FP8Q_F16; }
bool valid_fmt(int f) { return f == FP8Q_E4M3FN || f == FP8Q_E5M2; }
bool valid_act(int a) { return a == FP8Q_SILU || a == FP8Q_GELU || a == FP8Q_GELU_TANH; }
bool half_dtype(int dt) { return dt == FP8Q_BF16 || dt == FP8Q_F16; }
int64_t esize(int dt) { return dt == FP8Q_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t a) { return ((uintptr_t)p % (uintptr_t)a) == 0; }
int64_t blocks(int64_t n) { return n / 128 + (n % 128 != 0); }

struct Buf {
    const void* p;
    int64_t bytes;
};

bool overlap(const Buf& a, const Buf& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

// the first `outs` buffers are outputs: none may meet any other buffer
bool bad_overlap(const Buf* b, int n, int outs) {
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(b[i], b[j])) return true;
    return false;
}

fp8q_status_t launched() { return hipGetLastError() == hipSuccess ? FP8Q_OK : FP8Q_EHIP; }
hipStream_t S(void* s) { return (hipStream_t)s; }

// [rows, K] codes with their scales
struct Codes {
    const uint8_t* q;
    const float* s;
    int64_t rows, scale_rows;
};

// sizes of the products: M rows, N columns, K contraction
fp8q_status_t check_sizes(int64_t M, int64_t N, int64_t K, int64_t max_m) {
    if (M < 0 || N < 0 || K < 0) return FP8Q_EINVAL;
    if (K % 128 != 0) return FP8Q_ESHAPE;
    if (M > max_m || N > kMaxDim || K > kMaxDim) return FP8Q_EINVAL;
    return FP8Q_OK;
}

fp8q_status_t check_codes(const Codes& c, int64_t K) {
    if (c.rows == 0 || K == 0) return FP8Q_OK;
    if (!c.q || !c.s) return FP8Q_EINVAL;
    return aligned(c.q, 16) && aligned(c.s, 4) ? FP8Q_OK : FP8Q_EALIGN;
}

fp8q_status_t check_ws(const void* ws, int64_t bytes) {
    if (bytes == 0) return FP8Q_OK;
    if (!ws) return FP8Q_EINVAL;
    return aligned(ws, 256) ? FP8Q_OK : FP8Q_EALIGN;
}

constexpr int64_t kMaxFwdRows = int64_t(1) << 31;
// no tiling of an [M, N] product has more tiles than this
bool grid_ok(int64_t M, int64_t N) { return (M / 64 + 1) * (N / 128 + 1) <= kMaxTiles; }

fp8q_status_t forward(fp8q::MmFwd& f, int64_t M, int64_t N, int64_t K, bool gated, void* stream) {
    if (!valid_fmt(f.xfmt) || !valid_fmt(f.wfmt) || (f.y && !valid_dtype(f.ydt)) || (f.z && !valid_dtype(f.zdt)))
        return FP8Q_EDTYPE;
    fp8q_status_t st = check_sizes(M, N, K, kMaxFwdRows);
    if (st != FP8Q_OK) return st;
    if (!grid_ok(M, N)) return FP8Q_EINVAL;
    if (M == 0 || N == 0) return FP8Q_OK;
    const Codes x{f.x, f.xs, M, M}, w0{f.w0, f.ws0, N, blocks(N)}, w1{f.w1, f.ws1, gated ? N : 0, blocks(N)};
    for (const Codes* c : {&x, &w0, &w1}) {
        st = check_codes(*c, K);
        if (st != FP8Q_OK) return st;
    }
    if ((f.y && !aligned(f.y, esize(f.ydt))) || (f.z && !aligned(f.z, esize(f.zdt))) || (f.sinv && !aligned(f.sinv, 4)))
        return FP8Q_EALIGN;
    const int64_t wsb = fp8q::mm_fwd_workspace(M, N, K, gated, f.q != nullptr);
    st = check_ws(f.ws, wsb);
    if (st != FP8Q_OK) return st;
    const int64_t KB = K / 128;
    const Buf b[] = {{f.y, f.y ? M * N * esize(f.ydt) : 0},
                     {f.z, f.z ? 2 * M * N * esize(f.zdt) : 0},
                     {f.q, M * N},
                     {f.sinv, 4 * M * (N / 128)},
                     {f.ws, wsb},
                     {f.x, M * K},
                     {f.xs, 4 * M * KB},
                     {f.w0, N * K},
                     {f.ws0, 4 * blocks(N) * KB},
                     {f.w1, N * K},
                     {f.ws1, 4 * blocks(N) * KB}};
    if (bad_overlap(b, 11, 5)) return FP8Q_EINVAL;
    f.M = M;
    f.N = (int)N;
    f.K = (int)K;
    f.gated = gated;
    fp8q::launch_mm_fwd(f, S(stream));
    return launched();
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// norm
// ---------------------------------------------------------------------------

static fp8q_status_t norm_cast(bool group, const void* x, fp8q_dtype_t xdtype, const void* residual,
                               const void* weight, fp8q_dtype_t wdtype, int64_t rows, int64_t cols, float eps,
                               fp8q_fmt_t fmt, uint8_t* q, float* scale_inv, void* h, float* rstd, void* stream) {
    if (!valid_dtype(xdtype) || !valid_fmt(fmt) || (wdtype != xdtype && wdtype != FP8Q_F32)) return FP8Q_EDTYPE;
    if (rows < 0 || cols < 0) return FP8Q_EINVAL;
    if (group && cols % 128 != 0) return FP8Q_ESHAPE;
    if (rows > kMaxNormRows || cols > kMaxNormCols) return FP8Q_EINVAL;
    const int64_t n = rows * cols, es = esize(xdtype), sc = group ? rows * (cols / 128) : rows;
    if (rows == 0) return FP8Q_OK;
    if ((n > 0 && (!x || !weight || !q)) || (sc > 0 && !scale_inv)) return FP8Q_EINVAL;
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(h, es) || !aligned(weight, esize(wdtype)) ||
        !aligned(scale_inv, 4) || !aligned(rstd, 4))
        return FP8Q_EALIGN;
    // h may be x or the residual; otherwise the outputs meet nothing
    const Buf in_x{x, h == x ? 0 : n * es}, in_r{residual, h == residual ? 0 : n * es};
    const Buf b[] = {{q, n}, {scale_inv, 4 * sc}, {rstd, rstd ? 4 * rows : 0}, {h, n * es}, in_x, in_r,
                     {weight, cols * esize(wdtype)}};
    if (bad_overlap(b, 7, 4)) return FP8Q_EINVAL;
    if (cols == 0) {
        if (!group) fp8q::launch_fill_f32(scale_inv, rows, 1.0f, S(stream));
        return group ? FP8Q_OK : launched();
    }
    fp8q::launch_rmsnorm_cast(group, x, xdtype, residual, weight, wdtype, rows, cols, eps, fmt, q, scale_inv, h, rstd,
                              S(stream));
    return launched();
}

fp8q_status_t fp8q_rmsnorm_cast_group128(const void* x, fp8q_dtype_t xdtype, const void* residual, const void* weight,
                                         fp8q_dtype_t wdtype, int64_t rows, int64_t cols, float eps, fp8q_fmt_t fmt,
                                         uint8_t* q, float* scale_inv, void* h, float* rstd, void* stream) {
    return norm_cast(true, x, xdtype, residual, weight, wdtype, rows, cols, eps, fmt, q, scale_inv, h, rstd, stream);
}

fp8q_status_t fp8q_rmsnorm_cast_per_channel(const void* x, fp8q_dtype_t xdtype, const void* residual,
                                            const void* weight, fp8q_dtype_t wdtype, int64_t rows, int64_t cols,
                                            float eps, fp8q_fmt_t fmt, uint8_t* q, float* scale_inv, void* h,
                                            float* rstd, void* stream) {
    return norm_cast(false, x, xdtype, residual, weight, wdtype, rows, cols, eps, fmt, q, scale_inv, h, rstd, stream);
}

size_t fp8q_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows > kMaxNormRows || cols > kMaxNormCols) return 0;
    return (size_t)(fp8q::rmsnorm_bwd_parts(rows) * cols * 4);
}

fp8q_status_t fp8q_rmsnorm_backward(const void* dy, const void* h, fp8q_dtype_t dtype, const void* weight,
                                    fp8q_dtype_t wdtype, const float* rstd, const void* dh, int64_t rows, int64_t cols,
                                    void* dx, void* dweight, void* workspace, void* stream) {
    if (!valid_dtype(dtype) || (wdtype != dtype && wdtype != FP8Q_F32)) return FP8Q_EDTYPE;
    if (rows < 0 || cols < 0 || rows > kMaxNormRows || cols > kMaxNormCols) return FP8Q_EINVAL;
    const int64_t n = rows * cols, es = esize(dtype), we = esize(wdtype);
    if (cols == 0) return FP8Q_OK;
    if (n > 0 && (!dy || !h || !weight || !rstd || !dx)) return FP8Q_EINVAL;
    if (!aligned(dy, es) || !aligned(h, es) || !aligned(dh, es) || !aligned(dx, es) || !aligned(weight, we) ||
        !aligned(dweight, we) || !aligned(rstd, 4))
        return FP8Q_EALIGN;
    const int64_t wsb = dweight ? (int64_t)fp8q_rmsnorm_backward_workspace_bytes(rows, cols) : 0;
    const fp8q_status_t st = check_ws(workspace, wsb);
    if (st != FP8Q_OK) return st;
    const Buf b[] = {{dx, n * es}, {dweight, cols * we}, {workspace, wsb}, {dy, dx == dy ? 0 : n * es},
                     {dh, dx == dh ? 0 : n * es}, {h, n * es}, {weight, cols * we}, {rstd, 4 * rows}};
    // dx may be dy or dh, but then that tensor still may not meet another output
    if (bad_overlap(b, 8, 3)) return FP8Q_EINVAL;
    if (rows == 0) {
        if (dweight) {
            if (wdtype == FP8Q_F32) fp8q::launch_fill_f32((float*)dweight, cols, 0.0f, S(stream));
            else fp8q::launch_zero16(dweight, cols, S(stream));
            return launched();
        }
        return FP8Q_OK;
    }
    fp8q::launch_rmsnorm_bwd(dy, h, dtype, weight, wdtype, rstd, dh, rows, cols, dx, dweight, (float*)workspace,
                             S(stream));
    return launched();
}

// ---------------------------------------------------------------------------
// projections
// ---------------------------------------------------------------------------

static bool sizes_ok(int64_t M, int64_t N, int64_t K, int64_t max_m) {
    return check_sizes(M, N, K, max_m) == FP8Q_OK && M > 0 && N > 0;
}

size_t fp8q_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!sizes_ok(M, N, K, kMaxFwdRows)) return 0;
    return (size_t)fp8q::mm_fwd_workspace(M, N, K, false, false);
}

fp8q_status_t fp8q_linear(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w,
                          fp8q_fmt_t wfmt, const float* w_scale_inv, int64_t M, int64_t N, int64_t K, void* y,
                          fp8q_dtype_t ydtype, void* workspace, void* stream) {
    if (!valid_dtype(ydtype)) return FP8Q_EDTYPE;
    if (M > 0 && N > 0 && !y) return FP8Q_EINVAL;
    fp8q::MmFwd f{};
    f.x = x; f.xs = x_scale_inv; f.w0 = w; f.ws0 = w_scale_inv;
    f.xfmt = xfmt; f.wfmt = wfmt; f.y = y; f.ydt = ydtype; f.ws = workspace;
    return forward(f, M, N, K, false, stream);
}

size_t fp8q_gated_linear_workspace_bytes(int64_t M, int64_t F, int64_t K, int cast) {
    if (!sizes_ok(M, F, K, kMaxFwdRows)) return 0;
    return (size_t)fp8q::mm_fwd_workspace(M, F, K, true, cast != 0);
}

fp8q_status_t fp8q_gated_linear(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w_gate,
                                const float* w_gate_scale_inv, const uint8_t* w_up, const float* w_up_scale_inv,
                                fp8q_fmt_t wfmt, int64_t M, int64_t F, int64_t K, fp8q_act_t act, void* h,
                                fp8q_dtype_t hdtype, void* z, fp8q_dtype_t zdtype, void* workspace, void* stream) {
    if (!valid_dtype(hdtype) || !valid_act(act)) return FP8Q_EDTYPE;
    if (M > 0 && F > 0 && !h) return FP8Q_EINVAL;
    fp8q::MmFwd f{};
    f.x = x; f.xs = x_scale_inv; f.w0 = w_gate; f.ws0 = w_gate_scale_inv; f.w1 = w_up; f.ws1 = w_up_scale_inv;
    f.xfmt = xfmt; f.wfmt = wfmt; f.act = act; f.y = h; f.ydt = hdtype; f.z = z; f.zdt = zdtype; f.ws = workspace;
    return forward(f, M, F, K, true, stream);
}

fp8q_status_t fp8q_gated_linear_cast(const uint8_t* x, fp8q_fmt_t xfmt, const float* x_scale_inv,
                                     const uint8_t* w_gate, const float* w_gate_scale_inv, const uint8_t* w_up,
                                     const float* w_up_scale_inv, fp8q_fmt_t wfmt, int64_t M, int64_t F, int64_t K,
                                     fp8q_act_t act, fp8q_fmt_t fmt, uint8_t* q, float* scale_inv, void* z,
                                     fp8q_dtype_t zdtype, void* workspace, void* stream) {
    if (!valid_fmt(fmt) || !valid_act(act)) return FP8Q_EDTYPE;
    if (M < 0 || F < 0) return FP8Q_EINVAL;
    if (F % 128 != 0) return FP8Q_ESHAPE;
    if (M > 0 && F > 0 && (!q || !scale_inv)) return FP8Q_EINVAL;
    fp8q::MmFwd f{};
    f.x = x; f.xs = x_scale_inv; f.w0 = w_gate; f.ws0 = w_gate_scale_inv; f.w1 = w_up; f.ws1 = w_up_scale_inv;
    f.xfmt = xfmt; f.wfmt = wfmt; f.act = act; f.q = q; f.qfmt = fmt; f.sinv = scale_inv; f.z = z; f.zdt = zdtype;
    f.ws = workspace;
    return forward(f, M, F, K, true, stream);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

static fp8q_status_t backward(fp8q::MmBwd& f, int64_t M, int64_t N, int64_t K, bool gated, void* stream) {
    if (!half_dtype(f.dt) || !valid_fmt(f.xfmt) || !valid_fmt(f.wfmt) || (f.dwdt != f.dt && f.dwdt != FP8Q_F32))
        return FP8Q_EDTYPE;
    fp8q_status_t st = check_sizes(M, N, K, kMaxRows);
    if (st != FP8Q_OK) return st;
    if (!grid_ok(M, K) || !grid_ok(2 * N + 64, K)) return FP8Q_EINVAL;
    // the layout pass: 64 x 64 tiles of dy, 64 x 128 of the codes, 256 threads each
    const int64_t mt = M / 64 + 2, nt = N / 64 + 1;         // rows are padded to 64 or 128
    if (mt * nt + (K / 128) * (mt + 2 * nt) >= int64_t(1) << 24) return FP8Q_EINVAL;
    if (gated && (f.dw0 == nullptr) != (f.dw1 == nullptr) && N > 0 && K > 0) return FP8Q_EINVAL;
    const int64_t n = M * N;
    if (n > 0 && K > 0) {
        if (!f.dy || (gated && !f.z)) return FP8Q_EINVAL;
        const Codes x{f.x, f.xs, M, M}, w0{f.w0, f.ws0, N, 0}, w1{f.w1, f.ws1, gated ? N : 0, 0};
        for (const Codes* c : {&x, &w0, &w1}) {
            st = check_codes(*c, K);
            if (st != FP8Q_OK) return st;
        }
    }
    const int64_t we = esize(f.dwdt);
    if (!aligned(f.dy, 2) || !aligned(f.z, 2) || !aligned(f.dx, 2) || !aligned(f.dw0, we) || !aligned(f.dw1, we))
        return FP8Q_EALIGN;
    if (!f.dx && !f.dw0) return FP8Q_OK;
    const int64_t wsb = fp8q::mm_bwd_workspace(M, N, K, gated);
    st = check_ws(f.ws, wsb);
    if (st != FP8Q_OK) return st;
    const int64_t KB = K / 128;
    const Buf b[] = {{f.dx, M * K * 2}, {f.dw0, N * K * we}, {f.dw1, N * K * we}, {f.ws, wsb},
                     {f.dy, n * 2}, {f.z, 4 * n}, {f.x, M * K}, {f.xs, 4 * M * KB}, {f.w0, N * K},
                     {f.ws0, 4 * blocks(N) * KB}, {f.w1, N * K}, {f.ws1, 4 * blocks(N) * KB}};
    if (bad_overlap(b, 12, 4)) return FP8Q_EINVAL;
    if (K == 0 || (M == 0 && N == 0)) return FP8Q_OK;
    f.M = M;
    f.N = (int)N;
    f.K = (int)K;
    f.gated = gated;
    fp8q::launch_mm_bwd(f, S(stream));
    return launched();
}

size_t fp8q_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!sizes_ok(M, N, K, kMaxRows)) return 0;
    return (size_t)fp8q::mm_bwd_workspace(M, N, K, false);
}

fp8q_status_t fp8q_linear_backward(const void* dy, fp8q_dtype_t dtype, const uint8_t* x, fp8q_fmt_t xfmt,
                                   const float* x_scale_inv, const uint8_t* w, fp8q_fmt_t wfmt,
                                   const float* w_scale_inv, int64_t M, int64_t N, int64_t K, void* dx, void* dw,
                                   fp8q_dtype_t dwdtype, void* workspace, void* stream) {
    fp8q::MmBwd f{};
    f.dy = dy; f.dt = dtype; f.x = x; f.xs = x_scale_inv; f.w0 = w; f.ws0 = w_scale_inv;
    f.xfmt = xfmt; f.wfmt = wfmt; f.dx = dx; f.dw0 = dw; f.dwdt = dwdtype; f.ws = workspace;
    return backward(f, M, N, K, false, stream);
}

size_t fp8q_gated_linear_backward_workspace_bytes(int64_t M, int64_t F, int64_t K) {
    if (!sizes_ok(M, F, K, kMaxRows)) return 0;
    return (size_t)fp8q::mm_bwd_workspace(M, F, K, true);
}

fp8q_status_t fp8q_gated_linear_backward(const void* dp, const void* z, fp8q_dtype_t dtype, const uint8_t* x,
                                         fp8q_fmt_t xfmt, const float* x_scale_inv, const uint8_t* w_gate,
                                         const float* w_gate_scale_inv, const uint8_t* w_up,
                                         const float* w_up_scale_inv, fp8q_fmt_t wfmt, int64_t M, int64_t F, int64_t K,
                                         fp8q_act_t act, void* dx, void* dw_gate, void* dw_up, fp8q_dtype_t dwdtype,
                                         void* workspace, void* stream) {
    if (!valid_act(act)) return FP8Q_EDTYPE;
    fp8q::MmBwd f{};
    f.dy = dp; f.z = z; f.dt = dtype; f.x = x; f.xs = x_scale_inv; f.w0 = w_gate; f.ws0 = w_gate_scale_inv;
    f.w1 = w_up; f.ws1 = w_up_scale_inv; f.xfmt = xfmt; f.wfmt = wfmt; f.act = act;
    f.dx = dx; f.dw0 = dw_gate; f.dw1 = dw_up; f.dwdt = dwdtype; f.ws = workspace;
    return backward(f, M, F, K, true, stream);
}

}  // extern "C"
