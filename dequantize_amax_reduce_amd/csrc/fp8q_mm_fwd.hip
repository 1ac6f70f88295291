// fp8q_mm_fwd.hip -- the forward products on fp8 operands: one projection, or
// the gate and up projections with the activation and their product (and the
// group cast of it) in the same kernel.
//
// The kernels are in fp8q_mm_fwd.h.
#include "fp8q_mm_fwd.h"

namespace fp8q {

namespace {

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// enough for either kind of sum: the output types are not known here
int64_t mm_fwd_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool cast) {
    int64_t most = 0;
    for (int ex = cast ? 1 : 0; ex < 2; ++ex) {
        const Plan p = plan(M, N, K, gated, ex);
        const int64_t pb = cast && p.rows ? M * N * 4 : 0;
        most = std::max(most, up256(part_bytes(p, M, N, gated)) + pb);
    }
    return most;
}

void launch_mm_partial(const FwdArgs& a, int xfmt, int wfmt, const Plan& p, bool ex, hipStream_t st) {
    with_formats(xfmt, wfmt, [&](auto X, auto W) {
        with_tile(p, ex, [&](auto BM, auto EX) {
            k_mm<decltype(X)::value, decltype(W)::value, decltype(BM)::value, kOutPartial, decltype(EX)::value>
                <<<dim3((unsigned)(p.tm * p.tn), (unsigned)p.splits), kMmThreads, 0, st>>>(a);
        });
    });
}

void launch_mm_fwd(const MmFwd& f, hipStream_t st) {
    const bool gated = f.gated;
    const bool ex = f.M <= kExactMax || f.q || (f.y && f.ydt == kF32) || (f.z && f.zdt == kF32);
    const Plan p = plan(f.M, f.N, f.K, gated, ex);
    FwdArgs a{f.x, f.xs, f.w0, f.ws0, f.w1, f.ws1, f.M, f.N, f.K / 128, (uint32_t)p.tm, (uint32_t)p.tn, f.act,
              f.y, f.ydt, f.q, f.qfmt, f.sinv, f.z, f.zdt, 0, 0, gated, p.kper, nullptr, nullptr, 0, nullptr, 0};
    a.vec_y = f.N % 8 == 0 && (p.splits > 1 || al(f.y, 16));
    a.vec_z = f.N % 8 == 0 && al(f.z, 16);
    char* ws = (char*)f.ws;
    float* pbuf = nullptr;
    if (p.splits > 1) a.part = (float*)ws;
    if (f.q && p.rows) pbuf = (float*)ws;
    if (p.splits > 1)
        launch_mm_partial(a, f.xfmt, f.wfmt, p, ex, st);
    else
        with_formats(f.xfmt, f.wfmt, [&](auto X, auto W) {
            constexpr int XF = decltype(X)::value, WF = decltype(W)::value;
            if (p.rows) {
                if (gated) run_rows<XF, WF, kOutGated>(a, pbuf, st);
                else run_rows<XF, WF, kOutLinear>(a, pbuf, st);
                return;
            }
            with_tile(p, ex, [&](auto BM, auto EX) {
                const unsigned g = (unsigned)(p.tm * p.tn);
                if (gated) k_mm<XF, WF, decltype(BM)::value, kOutGated, decltype(EX)::value><<<g, kMmThreads, 0, st>>>(a);
                else k_mm<XF, WF, decltype(BM)::value, kOutLinear, decltype(EX)::value><<<g, kMmThreads, 0, st>>>(a);
            });
        });
    if (p.splits > 1) {
        const JoinArgs j{a.part, p.splits, f.M, f.N, gated, f.act, f.y, f.ydt, f.z, f.zdt, f.q, f.qfmt, f.sinv,
                         nullptr, 0, nullptr};
        const int V = f.N % 4 == 0 ? 4 : 1;
        const unsigned g = (unsigned)std::min<int64_t>((f.M * (f.N / V) + 255) / 256, 4096);
        if (f.q) k_mm_join<4, true><<<g, 256, 0, st>>>(j);
        else if (V == 4) k_mm_join<4, false><<<g, 256, 0, st>>>(j);
        else k_mm_join<1, false><<<g, 256, 0, st>>>(j);
    }
    if (pbuf) launch_group128_cast(pbuf, kF32, f.M * (f.N / 128), f.qfmt, f.q, f.sinv, st);
}

}  // namespace fp8q
