// Attention over the cache: Q8_0 blocks, f16 queries (kv_attention.h).
#include "kv_attention.h"

namespace qmv {

hipError_t kv_attention_q8_f16(const KvAttnArgs& a, const KvAttentionPlan& p, hipStream_t s) {
  return kv_attention_sizes<false, 1>(a, p, s);
}

}  // namespace qmv
