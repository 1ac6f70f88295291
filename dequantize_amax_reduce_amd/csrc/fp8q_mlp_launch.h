// fp8q_mlp_launch.h -- internal interface between the ABI layer of the layer
// norm and biased projections (argument validation) and their HIP launchers.
// Not installed; not part of the ABI.
#pragma once
#include "fp8q_ffn_launch.h"

namespace fp8q {

// what becomes of a norm's y
enum { kToPlain = 0, kToGroup = 1, kToRow = 2 };

struct LayerNorm {
    const void* x;
    int dt;
    const void* res;     // or nullptr
    const void* w;
    const void* b;       // or nullptr
    int wdt;
    int64_t rows, cols;
    float eps;
    int to, fmt;
    void* y;             // of dt (kToPlain), or codes of fmt
    float* sinv;
    void* h;             // or nullptr
    float* mean;         // or nullptr
    float* rstd;         // or nullptr
};
void launch_layernorm(const LayerNorm& a, hipStream_t st);

// partial sums of dweight and of dbias: 2 layernorm_bwd_parts(rows) rows of cols floats in ws
int64_t layernorm_bwd_parts(int64_t rows);
struct LayerNormBwd {
    const void* dy;
    const void* h;
    int dt;
    const void* w;
    int wdt;
    const float* mean;
    const float* rstd;
    const void* dh;      // or nullptr
    int64_t rows, cols;
    void* dx;
    void* dw;            // or nullptr
    void* db;            // or nullptr
    float* ws;
};
void launch_layernorm_bwd(const LayerNormBwd& a, hipStream_t st);

// out0[c] = sum of part[0 .. parts)[c] of cols floats each, in a fixed order;
// out1 likewise of the `parts` rows after those; either may be null
void launch_column_sums(const float* part, int64_t parts, int64_t cols, void* out0, void* out1, int dt, hipStream_t st);

// One projection with an epilogue: z = X W^T + bias (kept in f.z [M, N] where
// asked), then act(z) + res to f.y, or the group cast of act(z) to f.q.  f.w1,
// f.ws1 and f.gated are unused.
struct MmAct {
    MmFwd f;
    const void* bias;    // [N] of bdt, or nullptr
    int bdt;
    const void* res;     // [M, N] of f.ydt, or nullptr; may be f.y
};
int64_t mm_act_workspace(int64_t M, int64_t N, int64_t K, bool cast);
void launch_mm_act(const MmAct& a, hipStream_t st);

// Its backward: dz = dy act'(z), f.dx, f.dw0 and db, each or null (not all
// three); f.z is null where act is the identity.  f.w1, f.ws1, f.dw1 and f.gated
// are unused; any of f.M, f.N and f.K may be 0 (sums over nothing are zeros).
struct MmActBwd {
    MmBwd f;
    void* db;            // [N] of f.dwdt, or nullptr
};
int64_t mm_act_bwd_workspace(int64_t M, int64_t N, int64_t K);
void launch_mm_act_bwd(const MmActBwd& a, hipStream_t st);

}  // namespace fp8q
