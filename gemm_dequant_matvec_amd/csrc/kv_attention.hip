// Attention over the quantised cache: how a call is cut, the join of partial
// results, and the choice of the kernel's instance (kv_attention.h).
#include "kv_attention.h"

namespace qmv {
namespace {

constexpr int kThreads = 256;

// out = sum of 2^(ref_i - ref) o_i / sum of 2^(ref_i - ref) sum_i over a row's partial results, in
// their order, eight of them under way at a time.  A row has D / 4 threads.  Bound by memory: 96 tokens
// of 32 heads of 128 with 22 parts take 8 us, 4.2 TB/s.
template <int E>
__global__ __launch_bounds__(kThreads) void kv_join_kernel(const KvAttnArgs a) {
  constexpr int kAhead = 8;
  const int D = 32 * a.kv.nb, per = D >> 2, rows = kThreads / per;
  const int mine = threadIdx.x / per, x = threadIdx.x - mine * per;
  const int64_t end = int64_t(kv_row_start(a.kv, a.kv.B)) * a.q_heads;
  if (mine >= rows) return;
  const int64_t first = int64_t(kv_row_start(a.kv, 0)) * a.q_heads + mine;
  for (int64_t row = first + int64_t(blockIdx.x) * rows; row < end; row += int64_t(gridDim.x) * rows) {
    const int token = int(row / a.q_heads), h = int(row - int64_t(token) * a.q_heads);
    const float2* st = a.stats + row * a.slots;
    const float* sums = a.sums + row * a.slots * D + 4 * x;
    f32x4 o = {0, 0, 0, 0};
    float ref = -kInf, sum = 0.0f;
    for (int i0 = 0; i0 < a.slots; i0 += kAhead) {
      float2 s[kAhead];
      f32x4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = min(i0 + i, a.slots - 1);
        s[i] = st[at];
        v[i] = *reinterpret_cast<const f32x4*>(sums + int64_t(at) * D);
      }
      float next = ref;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next = fmaxf(next, s[i].x);
      const float from = next == -kInf ? 0.0f : next, f = __builtin_amdgcn_exp2f(ref - from);
      ref = next;
      sum *= f;
      o *= f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i0 + i >= a.slots || s[i].y == 0.0f) continue;  // what saw nothing has no values
        const float g = __builtin_amdgcn_exp2f(s[i].x - from);
        sum = fmaf(s[i].y, g, sum);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = fmaf(v[i][r], g, o[r]);
      }
    }
    if (a.lse && x == 0) a.lse[row] = sum == 0.0f ? -kInf : 0.69314718f * (ref + __builtin_amdgcn_logf(sum));
    f32x4 v = o * (1.0f / sum);
    if (sum == 0.0f) v = f32x4{0, 0, 0, 0};
    const int64_t to = token * a.out_token + h * a.out_head + 4 * x;
    if constexpr (E == 0) {
      __builtin_memcpy(static_cast<float*>(a.out) + to, &v, 16);
    } else {
      const u32x2 w = {pack16<E == 1>(v[0], v[1]), pack16<E == 1>(v[2], v[3])};
      __builtin_memcpy(static_cast<uint16_t*>(a.out) + to, &w, 8);
    }
  }
}

// How many parts to cut `tokens` into for `items` workgroups otherwise: up to two workgroups per
// unit, of `least` tokens at least; beyond that parts of 2048 tokens, which even out sequences of
// different lengths, up to eight workgroups per place.  (Parts of a prefix of 8200 tokens with 24 items:
// 21 of them 96 us the call, 10 of them 123, 5 of them 188.)
int parts(int64_t items, int64_t tokens, int least) {
  const int64_t fill = std::min(512 / items, (tokens + least - 1) / least);
  const int64_t even = std::min((tokens + 2047) / 2048, (4096 + items - 1) / items);
  return int(std::max<int64_t>({1, std::min<int64_t>(fill, 64), std::min<int64_t>(even, 64)}));
}

}  // namespace

KvAttentionPlan kv_attention_plan(const qmv_kv_cache& c, const qmv_kv_batch& b, const qmv_kv_attention_args& a) {
  KvAttentionPlan p{};
  const int64_t group = a.q_heads / c.heads, longest = std::min<int64_t>(a.max_kv, b.columns * c.page);
  auto cut = [&](int64_t rows, int64_t sequences, int64_t tokens, bool& many, int& blocks, int& splits) {
    // Up to four blocks of the kernel for few rows, which read the same tokens, beat one of the kernel for many.
    // 8 sequences of 4000 tokens, 8 heads of 128, Q8_0, bf16, a call in us with 32 / 64 / 96 / 128 rows of a head: 28
    // / 41 / 62 / 74, with the other kernel 41 / 48 / 51 / 55 (Q4_0, f16: 29 / 46 / 59 / 76 and 49 / 59 / 62 / 67).
    many = rows > 64 && c.heads * sequences <= 1 << 22;  // up to 512 threads each, counted in 32 bits
    const int per = many ? kManyRows : 16;
    blocks = int(std::min<int64_t>((rows + per - 1) / per, 65535));
    // blocks that have rows: no more than all rows fill, and one that begins in each sequence
    splits = parts(c.heads * std::min(sequences * blocks, b.T * group / per + sequences), tokens,
                   16 * (many ? kLeastMany : kLeastFew));
  };
  const int64_t q = std::min(a.max_q, b.T);
  int64_t own = std::max<int64_t>(1, longest - a.prefix);
  if (a.window) own = std::min(own, a.window + q);
  cut(q * group, b.B, own, p.many, p.row_blocks, p.splits);
  if (a.prefix) {
    cut(b.T * group, 1, std::min(longest, a.prefix), p.prefix_many, p.prefix_row_blocks, p.prefix_splits);
    p.slots = p.prefix_splits + p.splits;
  } else {
    p.slots = p.splits > 1 ? p.splits : 0;
  }
  const int64_t parts = b.T * a.q_heads * p.slots;
  p.sums_bytes = parts * c.D * 4;
  p.bytes = p.sums_bytes + (parts * 8 + 15) / 16 * 16;
  return p;
}

hipError_t launch_kv_attention(const qmv_kv_cache& c, const qmv_kv_batch& b, const qmv_kv_attention_args& t,
                               const KvAttentionPlan& plan, uint8_t* ws, hipStream_t s) {
  KvAttnArgs a{};
  a.kv = kv_args(c, b);
  a.q = t.q;
  a.out = t.out;
  a.lse = t.lse;
  a.sums = reinterpret_cast<float*>(ws);
  a.stats = reinterpret_cast<float2*>(ws + plan.sums_bytes);
  a.q_token = t.q_token, a.q_head = t.q_head, a.out_token = t.out_token, a.out_head = t.out_head;
  a.scale = t.scale * 1.44269504f;
  a.group = int(t.q_heads / c.heads);
  a.q_heads = int(t.q_heads);
  // past the longest sequence a window hides nothing and a prefix shares everything
  a.window = int(std::min<int64_t>(t.window, int64_t(1) << 30));
  a.prefix = int(std::min<int64_t>(t.prefix, b.columns * c.page));
  a.slots = plan.slots;
  const bool q4 = c.fmt == QMV_Q4_0;
  hipError_t e;
  if (t.dtype == QMV_F32) e = q4 ? kv_attention_q4_f32(a, plan, s) : kv_attention_q8_f32(a, plan, s);
  else if (t.dtype == QMV_F16) e = q4 ? kv_attention_q4_f16(a, plan, s) : kv_attention_q8_f16(a, plan, s);
  else e = q4 ? kv_attention_q4_bf16(a, plan, s) : kv_attention_q8_bf16(a, plan, s);
  if (e != hipSuccess || !plan.slots) return e;
  const int per_block = kThreads / int(c.D / 4);
  const dim3 grid(unsigned(std::min<int64_t>((b.T * t.q_heads + per_block - 1) / per_block, 1 << 22)));
  if (t.dtype == QMV_F32) hipLaunchKernelGGL((kv_join_kernel<0>), grid, dim3(kThreads), 0, s, a);
  else if (t.dtype == QMV_F16) hipLaunchKernelGGL((kv_join_kernel<1>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((kv_join_kernel<2>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace qmv
