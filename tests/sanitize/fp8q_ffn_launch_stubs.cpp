// Host-only stand-ins for the launchers of the feed-forward operators
// (fp8q_ffn_launch.h), for the sanitizer build of fp8q_ffn_abi.cpp.  Each
// checks the preconditions that the ABI layer promises and counts its calls.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdlib.h>

#include "fp8q_ffn_launch.h"

namespace {
long g_calls = 0;
void need(bool ok) {
    if (!ok) abort();
}
bool al(const void* p, uintptr_t a) { return (uintptr_t)p % a == 0; }
}  // namespace

extern "C" long fp8q_ffn_stub_count(void) { return g_calls; }
extern "C" void fp8q_ffn_stub_reset(void) { g_calls = 0; }

hipError_t hipGetLastError(void) { return hipSuccess; }

namespace fp8q {

void launch_fill_f32(float* p, int64_t n, float, hipStream_t) { need(p && n > 0); ++g_calls; }
void launch_zero16(void* p, int64_t n, hipStream_t) { need(p && n > 0); ++g_calls; }

void launch_rmsnorm_cast(bool group, const void* x, int, const void*, const void* w, int, int64_t rows, int64_t cols,
                         float, int, uint8_t* q, float* sinv, void*, float*, hipStream_t) {
    need(x && w && q && sinv && rows > 0 && cols > 0 && (!group || cols % 128 == 0));
    ++g_calls;
}

int64_t rmsnorm_bwd_parts(int64_t rows) { return rows < 512 ? rows : 512; }

void launch_rmsnorm_bwd(const void* dy, const void* h, int, const void* w, int, const float* rstd, const void*,
                        int64_t rows, int64_t cols, void* dx, void* dw, float* ws, hipStream_t) {
    need(dy && h && w && rstd && dx && rows > 0 && cols > 0 && (!dw || (ws && al(ws, 256))));
    ++g_calls;
}

int64_t mm_fwd_workspace(int64_t M, int64_t N, int64_t, bool gated, bool cast) {
    need(M > 0 && N > 0);
    return cast && M <= 64 ? M * N * 4 : M <= 200 ? 4 * M * N * (gated ? 8 : 4) : 0;
}

void launch_mm_fwd(const MmFwd& a, hipStream_t) {
    need(a.M > 0 && a.N > 0 && a.K >= 0 && a.K % 128 == 0);
    need(a.K == 0 || (a.x && a.xs && a.w0 && a.ws0 && al(a.x, 16) && al(a.w0, 16)));
    need(!a.gated || a.K == 0 || (a.w1 && a.ws1 && al(a.w1, 16)));
    need((a.y != nullptr) != (a.q != nullptr));
    need(!a.q || (a.sinv && a.gated && a.N % 128 == 0));
    ++g_calls;
}

int64_t mm_bwd_workspace(int64_t M, int64_t N, int64_t K, bool gated) {
    return M && N && K ? (gated ? 2 << 20 : 1 << 20) : 0;
}

void launch_mm_bwd(const MmBwd& a, hipStream_t) {
    need(a.M >= 0 && a.N >= 0 && a.K > 0 && a.K % 128 == 0 && (a.dx || a.dw0));
    need((a.dt == kBF16 || a.dt == kF16) && (a.dwdt == a.dt || a.dwdt == kF32));
    if (a.M > 0 && a.N > 0) {
        need(a.dy && a.x && a.xs && a.w0 && a.ws0 && a.ws && al(a.x, 16) && al(a.w0, 16) && al(a.ws, 256));
        need(!a.gated || (a.z && a.w1 && a.ws1 && (a.dw0 != nullptr) == (a.dw1 != nullptr)));
    }
    ++g_calls;
}

}  // namespace fp8q
