// fp8q_mm_act.hip -- a projection on fp8 operands with bias, activation and
// residual in its epilogue, or with the group cast of the activation.
//
//   z = X W^T + b;  y = act(z) + r, or q, scale_inv = cast(act(z))
//
// The kernels are in fp8q_mm_fwd.h: the epilogue runs where the tile's sums are
// in registers (k_mm), where the splits of a contraction are joined
// (k_mm_join), or where the waves' sums of few rows meet (k_mm_rows).
#include "fp8q_mlp_launch.h"
#include "fp8q_mm_act.h"

namespace fp8q {

template void launch_mm_act_whole<kE4M3>(const FwdArgs&, float*, int, const PlanAct&, bool, hipStream_t);

namespace {

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Sums are binary32 where an output shows them (a binary32 y or z, or a cast with
// its scales), and of up to 64 rows, as fp8q_linear's are: the weights' bytes bound
// those, and the fp8 instruction would take 3 us off 48 rows 18432 -> 7168 (28.8).
bool exact_sums(const MmFwd& f) {
    return f.M <= kExactMax || f.q || (f.y && f.ydt == kF32) || (f.z && f.zdt == kF32);
}

}  // namespace

// enough for either kind of sum: the output types are not known here
int64_t mm_act_workspace(int64_t M, int64_t N, int64_t K, bool cast) {
    int64_t most = 0;
    for (int ex = cast || M <= kExactMax ? 1 : 0; ex < 2; ++ex) {
        const Plan p = plan_act(M, N, K, ex).p;
        most = std::max(most, p.rows ? (cast ? M * N * 4 : 0) : up256(part_bytes(p, M, N, false)));
    }
    return most;
}

void launch_mm_act(const MmAct& e, hipStream_t st) {
    const MmFwd& f = e.f;
    const bool ex = exact_sums(f);
    const PlanAct pa = plan_act(f.M, f.N, f.K, ex);
    const Plan& p = pa.p;
    // a cast of up to 16 rows goes through binary32 values in the workspace: a
    // workgroup of k_mm_rows has no whole group of 128 columns
    float* pbuf = f.q && p.rows ? (float*)f.ws : nullptr;
    const FwdArgs a{f.x, f.xs, f.w0, f.ws0, nullptr, nullptr, f.M, f.N, f.K / 128, (uint32_t)p.tm, (uint32_t)p.tn, f.act,
                    f.y, f.ydt, f.q, f.qfmt, f.sinv, f.z, f.zdt, f.N % 8 == 0, 0, 0, p.kper, (float*)f.ws,
                    e.bias, e.bdt, e.res, (uint32_t)pa.tn2};
    if (p.splits > 1) launch_mm_partial(a, f.xfmt, f.wfmt, p, ex, st);
    else if (f.xfmt == kE4M3) launch_mm_act_whole<kE4M3>(a, pbuf, f.wfmt, pa, ex, st);
    else launch_mm_act_whole<kE5M2>(a, pbuf, f.wfmt, pa, ex, st);
    if (p.splits > 1) {
        const JoinArgs j{a.part, p.splits, f.M, f.N, 0, f.act, f.y, f.ydt, f.z, f.zdt, f.q, f.qfmt, f.sinv, e.bias, e.bdt, e.res};
        const int V = f.N % 4 == 0 ? 4 : 1;
        const unsigned g = (unsigned)std::min<int64_t>((f.M * (f.N / V) + 255) / 256, 4096);
        if (f.q) k_mm_join<4, true, true><<<g, 256, 0, st>>>(j);
        else if (V == 4) k_mm_join<4, false, true><<<g, 256, 0, st>>>(j);
        else k_mm_join<1, false, true><<<g, 256, 0, st>>>(j);
    }
    if (pbuf) launch_group128_cast(pbuf, kF32, f.M * (f.N / 128), f.qfmt, f.q, f.sinv, st);
}

}  // namespace fp8q
