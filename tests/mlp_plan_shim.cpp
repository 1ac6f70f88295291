// C entry points over csrc/fp8q_ffn_plan.h, for tests/mlp_plans.py.
#include "fp8q_ffn_plan.h"

extern "C" void shim_layernorm(int64_t rows, int64_t nv, int tiny, int64_t* o) {
    const fp8q::NormPlan p = fp8q::layernorm_plan(rows, nv, tiny != 0);
    o[0] = p.wave;
    o[1] = p.V;
    o[2] = p.threads;
    o[3] = p.at_once;
}

// vectors a thread (0: in passes), threads, workgroups
extern "C" void shim_layernorm_bwd(int64_t rows, int64_t nv, int64_t* o) {
    const fp8q::NormPlan p = fp8q::norm_bwd_plan(rows, nv);
    o[0] = p.V;
    o[1] = p.threads;
    o[2] = p.groups;
}

// rows a tile (0: few rows), splits, blocks of 128 a split, row tiles, column tiles of 256, of 64 nt2, nt2
extern "C" void shim_act(int64_t M, int64_t N, int64_t K, int ex, int64_t* o) {
    const fp8q::PlanAct a = fp8q::plan_act(M, N, K, ex != 0);
    o[0] = a.p.rows ? 0 : a.p.bm;
    o[1] = a.p.splits;
    o[2] = a.p.kper;
    o[3] = a.p.tm;
    o[4] = a.p.tn;
    o[5] = a.tn2;
    o[6] = a.nt2;
}
extern "C" double shim_mixed_rounds(int64_t whole, int64_t part, double r) { return fp8q::mixed_rounds(whole, part, r); }

// of dx, then of dw: rows a tile, splits, steps a split; then whether one launch has both
extern "C" void shim_bwd_act(int64_t M, int64_t N, int64_t K, int rest, int64_t* o) {
    const fp8q::PlanBwd p = fp8q::plan_bwd_act(M, N, K, rest != 0);
    for (const fp8q::Plan16* q : {&p.dx, &p.dw}) {
        *o++ = q->bm;
        *o++ = q->splits;
        *o++ = q->kper;
    }
    *o = p.both;
}

// rows a tile of dx and of dw where a joint launch's products are asked for alone
extern "C" void shim_bwd_alone(int64_t M, int64_t N, int64_t K, int rest, int64_t* o) {
    const fp8q::PlanBwd p = fp8q::plan_bwd_act(M, N, K, rest != 0);
    o[0] = fp8q::alone16(M, K, p.dx.kper).bm;
    o[1] = fp8q::alone16(N, K, p.dw.kper).bm;
}
extern "C" double shim_time16(int64_t M, int64_t N, int64_t steps, int bm) {
    return fp8q::time16(fp8q::Plan16{bm, 1, (int)steps, 0}, M, N);
}
