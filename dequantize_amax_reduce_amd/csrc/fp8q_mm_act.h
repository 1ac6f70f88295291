// fp8q_mm_act.h -- launches of the projection with an epilogue, by the format of
// x: fp8q_mm_act.hip compiles those of e4m3fn, fp8q_mm_act_e5m2.hip the others.
#pragma once
#include "fp8q_mm_fwd.h"

namespace fp8q {

// every product but a split one
template <int XF> void launch_mm_act_whole(const FwdArgs& a, float* pbuf, int wfmt, const PlanAct& p, bool ex, hipStream_t st) {
    auto go = [&](auto W) {
        constexpr int WF = decltype(W)::value;
        if (p.p.rows) return run_rows<XF, WF, kOutAct>(a, pbuf, st);
        const unsigned g = (unsigned)(p.p.tm * (p.p.tn + p.tn2));
        if (ex) {
            if (p.nt2 == 2) k_mm_act<XF, WF, 64, 2, true><<<g, kMmThreads, 0, st>>>(a);
            else if (p.p.bm == 128) k_mm_act<XF, WF, 128, 4, true><<<g, kMmThreads, 0, st>>>(a);
            else k_mm_act<XF, WF, 64, 4, true><<<g, kMmThreads, 0, st>>>(a);
        } else {
            if (p.nt2 == 2) k_mm_act<XF, WF, 64, 2, false><<<g, kMmThreads, 0, st>>>(a);
            else if (p.nt2 == 3) k_mm_act<XF, WF, 256, 3, false><<<g, kMmThreads, 0, st>>>(a);
            else if (p.p.bm == 256) k_mm_act<XF, WF, 256, 4, false><<<g, kMmThreads, 0, st>>>(a);
            else if (p.p.bm == 128) k_mm_act<XF, WF, 128, 4, false><<<g, kMmThreads, 0, st>>>(a);
            else k_mm_act<XF, WF, 64, 4, false><<<g, kMmThreads, 0, st>>>(a);
        }
    };
    if (wfmt == kE4M3) go(KC<kE4M3>{});
    else go(KC<kE5M2>{});
}
extern template void launch_mm_act_whole<kE4M3>(const FwdArgs&, float*, int, const PlanAct&, bool, hipStream_t);
extern template void launch_mm_act_whole<kE5M2>(const FwdArgs&, float*, int, const PlanAct&, bool, hipStream_t);

}  // namespace fp8q
