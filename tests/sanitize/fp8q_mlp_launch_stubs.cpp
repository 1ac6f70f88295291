// Host-only stand-ins for the launchers of layer norm and biased projections
// (fp8q_mlp_launch.h), for the sanitizer build of fp8q_mlp_abi.cpp.  Each checks
// the preconditions that the ABI layer promises and counts its calls.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdlib.h>

#include "fp8q_mlp_launch.h"

namespace {
long g_calls = 0;
void need(bool ok) {
    if (!ok) abort();
}
bool al(const void* p, uintptr_t a) { return (uintptr_t)p % a == 0; }
}  // namespace

extern "C" long fp8q_mlp_stub_count(void) { return g_calls; }
extern "C" void fp8q_mlp_stub_reset(void) { g_calls = 0; }

hipError_t hipGetLastError(void) { return hipSuccess; }

namespace fp8q {

void launch_fill_f32(float* p, int64_t n, float, hipStream_t) { need(p && n > 0); ++g_calls; }
void launch_zero16(void* p, int64_t n, hipStream_t) { need(p && n > 0); ++g_calls; }

void launch_layernorm(const LayerNorm& a, hipStream_t) {
    need(a.x && a.w && a.y && a.rows > 0 && a.cols > 0);
    need(a.to == kToPlain || (a.sinv && (a.to == kToRow || a.cols % 128 == 0)));
    ++g_calls;
}

int64_t layernorm_bwd_parts(int64_t rows) { return rows < 512 ? rows : 512; }

void launch_layernorm_bwd(const LayerNormBwd& a, hipStream_t) {
    need(a.dy && a.h && a.w && a.mean && a.rstd && a.dx && a.rows > 0 && a.cols > 0);
    need((!a.dw && !a.db) || (a.ws && al(a.ws, 256)));
    ++g_calls;
}

int64_t mm_act_workspace(int64_t M, int64_t N, int64_t, bool cast) {
    need(M > 0 && N > 0);
    return cast && M <= 64 ? M * N * 4 : M <= 200 ? 16 * M * N : 0;
}

void launch_mm_act(const MmAct& e, hipStream_t) {
    const MmFwd& a = e.f;
    need(a.M > 0 && a.N > 0 && a.K >= 0 && a.K % 128 == 0 && a.act >= 0 && a.act <= kRelu);
    need(a.K == 0 || (a.x && a.xs && a.w0 && a.ws0 && al(a.x, 16) && al(a.w0, 16)));
    need((a.y != nullptr) != (a.q != nullptr) && !(a.q && e.res));
    need(!a.q || (a.sinv && a.N % 128 == 0));
    ++g_calls;
}

int64_t mm_act_bwd_workspace(int64_t M, int64_t N, int64_t K) { return M && N ? (K ? 2 << 20 : 1 << 20) : 0; }

void launch_mm_act_bwd(const MmActBwd& e, hipStream_t) {
    const MmBwd& a = e.f;
    need(a.M >= 0 && a.N >= 0 && a.K >= 0 && a.K % 128 == 0 && (a.dx || a.dw0 || e.db));
    need((a.dt == kBF16 || a.dt == kF16) && (a.dwdt == a.dt || a.dwdt == kF32) && a.act >= 0 && a.act <= kRelu);
    if (a.M > 0 && a.N > 0) {
        need(a.dy && (a.z != nullptr) == (a.act != kIdentity) && a.ws && al(a.ws, 256));
        if (a.K > 0 && (a.dx || a.dw0)) need(a.x && a.xs && a.w0 && a.ws0 && al(a.x, 16) && al(a.w0, 16));
    }
    ++g_calls;
}

}  // namespace fp8q
