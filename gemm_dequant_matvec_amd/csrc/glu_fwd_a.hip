// Gated products of many tokens, formats W4A16_G64, Q4K, DENSE_BF16.
#include "glu_fwd.h"

namespace qmv {

hipError_t launch_glu_fwd_a(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s) {
  switch (fmt) {
    case QMV_W4A16_G64: return f16 ? glu_fwd_go<QMV_W4A16_G64, true>(p, s) : glu_fwd_go<QMV_W4A16_G64, false>(p, s);
    case QMV_Q4K: return f16 ? glu_fwd_go<QMV_Q4K, true>(p, s) : glu_fwd_go<QMV_Q4K, false>(p, s);
    case QMV_DENSE_BF16: return f16 ? glu_fwd_go<QMV_DENSE_BF16, true>(p, s) : glu_fwd_go<QMV_DENSE_BF16, false>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmv
