// Backward pass of the gated products, formats W4A16_G64, Q4K, DENSE_BF16.
#include "glu_bwd.h"

namespace qmv {

hipError_t launch_glu_bwd_a(int fmt, bool f16, const GluBwdArgs& p, const GluBwdPlan& plan, hipStream_t s) {
  switch (fmt) {
    case QMV_W4A16_G64: return f16 ? glu_bwd_go<QMV_W4A16_G64, true>(p, plan, s) : glu_bwd_go<QMV_W4A16_G64, false>(p, plan, s);
    case QMV_Q4K: return f16 ? glu_bwd_go<QMV_Q4K, true>(p, plan, s) : glu_bwd_go<QMV_Q4K, false>(p, plan, s);
    case QMV_DENSE_BF16: return f16 ? glu_bwd_go<QMV_DENSE_BF16, true>(p, plan, s) : glu_bwd_go<QMV_DENSE_BF16, false>(p, plan, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
