// C entry points over csrc/fp8q_ffn_plan.h, for tests/ffn_plans.py.
#include "fp8q_ffn_plan.h"

using namespace fp8q;

static void put16(const Plan16& p, int64_t* o) {
    o[0] = p.bm;
    o[1] = p.splits;
    o[2] = p.kper;
}
static void put_norm(const NormPlan& p, int64_t* o) {
    o[0] = p.wave;
    o[1] = p.V;
    o[2] = p.threads;
    o[3] = p.at_once;
}

extern "C" {
void shim_fwd(int64_t M, int64_t N, int64_t K, int gated, int ex, int64_t* o) {
    const Plan p = plan(M, N, K, gated != 0, ex != 0);
    o[0] = p.rows ? 0 : p.bm;
    o[1] = p.splits;
    o[2] = p.kper;
}
void shim_dx(int64_t M, int64_t N, int64_t K, int gated, int rest, int64_t* o) {
    put16(plan_dx(M, N, K, gated != 0, rest != 0), o);
}
void shim_dw(int64_t M, int64_t N, int64_t K, int gated, int rest, int64_t* o) {
    put16(plan_dw(M, N, K, gated != 0, rest != 0), o);
}
void shim_norm(int64_t rows, int64_t nv, int64_t* o) { put_norm(norm_plan(rows, nv), o); }
void shim_norm_bwd(int64_t rows, int64_t nv, int64_t* o) { put_norm(norm_bwd_plan(rows, nv), o); }
int64_t shim_exact_max() { return kExactMax; }
}
