// Backward pass of the gated products, formats Q8_0, Q6K, I8_ROW.
#include "glu_bwd.h"

namespace qmv {

hipError_t launch_glu_bwd_b(int fmt, bool f16, const GluBwdArgs& p, const GluBwdPlan& plan, hipStream_t s) {
  switch (fmt) {
    case QMV_Q8_0: return f16 ? glu_bwd_go<QMV_Q8_0, true>(p, plan, s) : glu_bwd_go<QMV_Q8_0, false>(p, plan, s);
    case QMV_Q6K: return f16 ? glu_bwd_go<QMV_Q6K, true>(p, plan, s) : glu_bwd_go<QMV_Q6K, false>(p, plan, s);
    case QMV_I8_ROW: return f16 ? glu_bwd_go<QMV_I8_ROW, true>(p, plan, s) : glu_bwd_go<QMV_I8_ROW, false>(p, plan, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
