// C entry point over csrc/fp8q_ffn_plan.h, for tests/mlp_plans.py.
#include "fp8q_ffn_plan.h"

extern "C" void shim_layernorm(int64_t rows, int64_t nv, int tiny, int64_t* o) {
    const fp8q::NormPlan p = fp8q::layernorm_plan(rows, nv, tiny != 0);
    o[0] = p.wave;
    o[1] = p.V;
    o[2] = p.threads;
    o[3] = p.at_once;
}
