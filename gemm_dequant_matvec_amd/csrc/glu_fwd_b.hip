// Gated products of many tokens, formats Q8_0, Q6K, I8_ROW.
#include "glu_fwd.h"

namespace qmv {

hipError_t launch_glu_fwd_b(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s) {
  switch (fmt) {
    case QMV_Q8_0: return f16 ? glu_fwd_go<QMV_Q8_0, true>(p, s) : glu_fwd_go<QMV_Q8_0, false>(p, s);
    case QMV_Q6K: return f16 ? glu_fwd_go<QMV_Q6K, true>(p, s) : glu_fwd_go<QMV_Q6K, false>(p, s);
    case QMV_I8_ROW: return f16 ? glu_fwd_go<QMV_I8_ROW, true>(p, s) : glu_fwd_go<QMV_I8_ROW, false>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
