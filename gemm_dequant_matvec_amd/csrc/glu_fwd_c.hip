// Gated products of many tokens, formats Q4_0, Q5_0, Q5K.
#include "glu_fwd.h"

namespace qmv {

hipError_t launch_glu_fwd_c(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s) {
  switch (fmt) {
    case QMV_Q4_0: return f16 ? glu_fwd_go<QMV_Q4_0, true>(p, s) : glu_fwd_go<QMV_Q4_0, false>(p, s);
    case QMV_Q5_0: return f16 ? glu_fwd_go<QMV_Q5_0, true>(p, s) : glu_fwd_go<QMV_Q5_0, false>(p, s);
    case QMV_Q5K: return f16 ? glu_fwd_go<QMV_Q5K, true>(p, s) : glu_fwd_go<QMV_Q5K, false>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
