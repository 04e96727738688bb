// Backward pass of the gated products, formats Q4_0, Q5_0, Q5K.
#include "glu_bwd.h"

namespace qmv {

hipError_t launch_glu_bwd_c(int fmt, bool f16, const GluBwdArgs& p, const GluBwdPlan& plan, hipStream_t s) {
  switch (fmt) {
    case QMV_Q4_0: return f16 ? glu_bwd_go<QMV_Q4_0, true>(p, plan, s) : glu_bwd_go<QMV_Q4_0, false>(p, plan, s);
    case QMV_Q5_0: return f16 ? glu_bwd_go<QMV_Q5_0, true>(p, plan, s) : glu_bwd_go<QMV_Q5_0, false>(p, plan, s);
    case QMV_Q5K: return f16 ? glu_bwd_go<QMV_Q5K, true>(p, plan, s) : glu_bwd_go<QMV_Q5K, false>(p, plan, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
