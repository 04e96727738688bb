// Internal declarations of the key / value cache (qmv_cache.h): its geometry on
// the device, the batch, and the launchers.
#pragma once

#include "../../include/qmv_cache.h"
#include "qmv_internal.h"

namespace qmv {

// A cache and the batch of a call, as the kernels take them.  A "group" is 4 tokens, a
// "set" the 16 tokens of one record of the layout.
struct KvArgs {
  uint8_t* data;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t stride;    // of the table
  int64_t page_bytes;  // of all heads
  int T, B, columns, pages, heads, nb;
  int head_bytes, set_bytes, sets;  // of a page's head; of a set; sets of a page
  uint32_t magic;    // u / sets = (u * magic) >> 32 for u < 2^26
};

inline int64_t kv_set_bytes(int fmt, int64_t D) { return D / 32 * (2 * (fmt == QMV_Q8_0 ? 512 : 256) + 64); }

inline KvArgs kv_args(const qmv_kv_cache& c, const qmv_kv_batch& b) {
  KvArgs a{};
  a.data = static_cast<uint8_t*>(c.data);
  a.q_start = b.q_start;
  a.kv_len = b.kv_len;
  a.table = b.table;
  a.stride = b.stride;
  a.T = int(b.T);
  a.B = int(b.B);
  a.columns = int(b.columns);
  a.pages = int(c.pages);
  a.heads = int(c.heads);
  a.nb = int(c.D / 32);
  a.sets = c.page / 16;
  a.set_bytes = int(kv_set_bytes(c.fmt, c.D));
  a.head_bytes = a.sets * a.set_bytes;
  a.page_bytes = c.heads * int64_t(a.head_bytes);
  a.magic = a.sets == 1 ? 0u : uint32_t((int64_t(1) << 32) / a.sets + 1);
  return a;
}

// How an attention call is cut: `row_blocks` workgroups share a sequence's rows (many: of the
// kernel for more than 64 of them), each sequence's tokens go to `splits`; the same for the
// shared prefix.  slots: partial results per row (0: the only workgroup of a row writes it).
struct KvAttentionPlan {
  bool many, prefix_many;
  int row_blocks, splits, prefix_row_blocks, prefix_splits;
  int slots;
  int64_t sums_bytes, bytes;  // partial sums, then a reference and a weight sum of each
};
KvAttentionPlan kv_attention_plan(const qmv_kv_cache& c, const qmv_kv_batch& b, const qmv_kv_attention_args& a);

// Launchers: hipSuccess or the launch error; arguments are already validated.
hipError_t launch_kv_write(const qmv_kv_cache& c, const qmv_kv_batch& b, const void* k, int64_t k_token, int64_t k_head,
                           const void* v, int64_t v_token, int64_t v_head, int dtype, hipStream_t s);
hipError_t launch_kv_read(const qmv_kv_cache& c, const qmv_kv_batch& b, void* k, int64_t k_token, int64_t k_head, void* v,
                          int64_t v_token, int64_t v_head, int dtype, hipStream_t s);
hipError_t launch_kv_attention(const qmv_kv_cache& c, const qmv_kv_batch& b, const qmv_kv_attention_args& a,
                               const KvAttentionPlan& plan, uint8_t* ws, hipStream_t s);

// ----------------------------------------------------------- device helpers

__device__ __forceinline__ int kv_row_start(const KvArgs& a, int b) { return min(max(a.q_start[b], 0), a.T); }

// Page index of set u and the set's place in it.
__device__ __forceinline__ int kv_page_of(const KvArgs& a, uint32_t u, int& set) {
  const uint32_t p = a.sets == 1 ? u : __umulhi(u, a.magic);
  set = int(u - p * uint32_t(a.sets));
  return int(p);
}

// The largest b with first(b) <= v (0 if there is none), by a whole wave: each step
// narrows 64 to 1, ends for any values, and stays within 0 .. B - 1.
template <class F>
__device__ __forceinline__ int kv_search(int B, int64_t v, F first) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 63) >> 6, at = lane * step;
    const bool in = at < n && int64_t(first(lo + min(at, n - 1))) <= v;
    const int skip = max(0, int(__popcll(__ballot(in))) - 1) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

}  // namespace qmv
