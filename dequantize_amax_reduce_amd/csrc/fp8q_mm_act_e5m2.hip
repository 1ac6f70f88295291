// fp8q_mm_act_e5m2.hip -- the projection with an epilogue of e5m2 activations, in
// a translation unit of its own, compiled in parallel.
#include "fp8q_mm_act.h"

namespace fp8q {

template void launch_mm_act_whole<kE5M2>(const FwdArgs&, float*, int, const PlanAct&, bool, hipStream_t);

}  // namespace fp8q
