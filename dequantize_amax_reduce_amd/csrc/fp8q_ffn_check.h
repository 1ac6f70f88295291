// fp8q_ffn_check.h -- argument checks that the ABI layers of the feed-forward
// operators share (fp8q_ffn_abi.cpp, fp8q_mlp_abi.cpp).  Host code only.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q_ffn.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 21;    // K, N, F
constexpr int64_t kMaxRows = 65535 * 64;         // M of a backward pass
constexpr int64_t kMaxNormRows = INT32_MAX, kMaxNormCols = int64_t(1) << 30;
constexpr int64_t kMaxTiles = (int64_t(1) << 23) - 1;   // workgroups of 512 threads: 2^32 threads a grid

inline bool valid_dtype(int dt) { return dt == FP8Q_F32 || dt == FP8Q_BF16 || dt == FP8Q_F16; }
inline bool valid_fmt(int f) { return f == FP8Q_E4M3FN || f == FP8Q_E5M2; }
inline bool valid_act(int a) { return a == FP8Q_SILU || a == FP8Q_GELU || a == FP8Q_GELU_TANH; }
inline bool valid_unary(int a) { return valid_act(a) || a == FP8Q_IDENTITY || a == FP8Q_RELU; }
inline bool half_dtype(int dt) { return dt == FP8Q_BF16 || dt == FP8Q_F16; }
inline int64_t esize(int dt) { return dt == FP8Q_F32 ? 4 : 2; }
inline bool aligned(const void* p, int64_t a) { return ((uintptr_t)p % (uintptr_t)a) == 0; }
inline int64_t blocks(int64_t n) { return n / 128 + (n % 128 != 0); }

struct Buf {
    const void* p;
    int64_t bytes;
};

inline bool overlap(const Buf& a, const Buf& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

// the first `outs` buffers are outputs: none may meet any other buffer
inline bool bad_overlap(const Buf* b, int n, int outs) {
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(b[i], b[j])) return true;
    return false;
}

inline fp8q_status_t launched() { return hipGetLastError() == hipSuccess ? FP8Q_OK : FP8Q_EHIP; }
inline hipStream_t S(void* s) { return (hipStream_t)s; }

// [rows, K] codes with their scales
struct Codes {
    const uint8_t* q;
    const float* s;
    int64_t rows, scale_rows;
};

// sizes of the products: M rows, N columns, K contraction
inline fp8q_status_t check_sizes(int64_t M, int64_t N, int64_t K, int64_t max_m) {
    if (M < 0 || N < 0 || K < 0) return FP8Q_EINVAL;
    if (K % 128 != 0) return FP8Q_ESHAPE;
    if (M > max_m || N > kMaxDim || K > kMaxDim) return FP8Q_EINVAL;
    return FP8Q_OK;
}

inline fp8q_status_t check_codes(const Codes& c, int64_t K) {
    if (c.rows == 0 || K == 0) return FP8Q_OK;
    if (!c.q || !c.s) return FP8Q_EINVAL;
    return aligned(c.q, 16) && aligned(c.s, 4) ? FP8Q_OK : FP8Q_EALIGN;
}

inline fp8q_status_t check_ws(const void* ws, int64_t bytes) {
    if (bytes == 0) return FP8Q_OK;
    if (!ws) return FP8Q_EINVAL;
    return aligned(ws, 256) ? FP8Q_OK : FP8Q_EALIGN;
}

constexpr int64_t kMaxFwdRows = int64_t(1) << 31;
// no tiling of an [M, N] product has more tiles than this
inline bool grid_ok(int64_t M, int64_t N) { return (M / 64 + 1) * (N / 128 + 1) <= kMaxTiles; }

inline bool sizes_ok(int64_t M, int64_t N, int64_t K, int64_t max_m) {
    return check_sizes(M, N, K, max_m) == FP8Q_OK && M > 0 && N > 0;
}

}  // namespace
