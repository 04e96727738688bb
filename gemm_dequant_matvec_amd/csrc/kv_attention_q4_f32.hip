// Attention over the cache: Q4_0 blocks, f32 queries (kv_attention.h).
#include "kv_attention.h"

namespace qmv {

hipError_t kv_attention_q4_f32(const KvAttnArgs& a, const KvAttentionPlan& p, hipStream_t s) {
  return kv_attention_sizes<true, 0>(a, p, s);
}

}  // namespace qmv
