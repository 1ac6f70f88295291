// fp8q_ffn_launch.h -- internal interface between the ABI layer of the
// feed-forward operators (argument validation) and their HIP launchers.
// Not installed; not part of the ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q_launch.h"

namespace fp8q {

enum { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

// All launchers enqueue on `st` and never synchronise.  Preconditions
// (checked by the ABI layer): sizes > 0 unless stated, pointers valid and
// aligned as the header says, outputs disjoint from inputs.

// n 16-bit zeros; a kernel, so that a captured call records no memset
void launch_zero16(void* p, int64_t n, hipStream_t st);

// group: scales per 128 columns (cols % 128 == 0), else per row
void launch_rmsnorm_cast(bool group, const void* x, int dt, const void* res, const void* w, int wdt, int64_t rows,
                         int64_t cols, float eps, int fmt, uint8_t* q, float* sinv, void* h, float* rstd,
                         hipStream_t st);
// partial sums of dweight: rmsnorm_bwd_parts(rows) rows of cols floats in ws
int64_t rmsnorm_bwd_parts(int64_t rows);
void launch_rmsnorm_bwd(const void* dy, const void* h, int dt, const void* w, int wdt, const float* rstd,
                        const void* dh, int64_t rows, int64_t cols, void* dx, void* dw, float* ws, hipStream_t st);

// The forward products: a projection or a gated pair.  K may be 0.
struct MmFwd {
    const uint8_t* x;
    const float* xs;
    const uint8_t* w0;   // the projection, or the gate
    const float* ws0;
    const uint8_t* w1;   // the up projection (gated)
    const float* ws1;
    int64_t M;
    int N, K;            // N: columns of the output (F for a gated pair)
    bool gated;
    int xfmt, wfmt, act;
    void* y;             // [M, N] of ydt, or nullptr with q
    int ydt;
    uint8_t* q;          // fp8 codes of the group cast with qfmt (gated, N % 128 == 0), or nullptr
    int qfmt;
    float* sinv;         // [M, N / 128]
    void* z;             // [M, 2 N] of zdt, or nullptr
    int zdt;
    void* ws;
};
int64_t mm_fwd_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool cast);
void launch_mm_fwd(const MmFwd& a, hipStream_t st);

// The backward products of a projection or a gated pair; dx or the weight
// gradients may be null; M or N may be 0 (zeros are written).
struct MmBwd {
    const void* dy;      // [M, N] of dt (kBF16 or kF16)
    const void* z;       // [M, 2 N] of dt, or nullptr
    int dt;
    const uint8_t* x;
    const float* xs;
    const uint8_t* w0;
    const float* ws0;
    const uint8_t* w1;
    const float* ws1;
    int64_t M;
    int N, K;
    bool gated;
    int xfmt, wfmt, act;
    void* dx;
    void* dw0;
    void* dw1;
    int dwdt;
    void* ws;
};
int64_t mm_bwd_workspace(int64_t M, int64_t N, int64_t K, bool gated);
void launch_mm_bwd(const MmBwd& a, hipStream_t st);

}  // namespace fp8q
