// Gated products of many tokens: dispatch, the elementwise half of the backward
// pass and the sum of its split partials.
#include <algorithm>

#include "glu_bwd.h"
#include "glu_fwd.h"

namespace qmv {

hipError_t launch_glu_fwd_a(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s);
hipError_t launch_glu_fwd_b(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s);
hipError_t launch_glu_fwd_c(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s);
hipError_t launch_glu_bwd_a(int fmt, bool f16, const GluBwdArgs& p, const GluBwdPlan& plan, hipStream_t s);
hipError_t launch_glu_bwd_b(int fmt, bool f16, const GluBwdArgs& p, const GluBwdPlan& plan, hipStream_t s);
hipError_t launch_glu_bwd_c(int fmt, bool f16, const GluBwdArgs& p, const GluBwdPlan& plan, hipStream_t s);

namespace {

constexpr int kThreads = 256;

// What rounding v (f32) to the 16-bit value `bits` left over, to be rounded to the
// same type: with it, v is kept to 16 (bf16) or 22 (f16) bits, and where f16 ends, to
// multiples of 2^-24.  Zero behind a value that is no longer finite: dX follows it.
template <bool F16>
__device__ __forceinline__ float left_over(float v, uint32_t bits) {
  const float r = v - unpack16<F16>(bits & 0xFFFFu);
  return fabsf(r) < __builtin_inff() ? r : 0.0f;
}

// Eight values: dG = dH U act'(G), dU = dH act(G); LOW: also the low parts of both.
template <bool F16, int ACT, bool LOW>
__device__ __forceinline__ void dgates8(u32x4 gv, u32x4 uv, u32x4 hv, u32x4& og, u32x4& ou, u32x4& lg, u32x4& lu) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a[2], b[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t gw = gv[i], uw = uv[i], hw = hv[i];
      float av, da;
      act_both<ACT>(unpack16<F16>(e ? gw >> 16 : gw & 0xFFFFu), av, da);
      const float d = unpack16<F16>(e ? hw >> 16 : hw & 0xFFFFu);
      a[e] = d * unpack16<F16>(e ? uw >> 16 : uw & 0xFFFFu) * da;
      b[e] = d * av;
    }
    og[i] = pack16<F16>(a[0], a[1]);
    ou[i] = pack16<F16>(b[0], b[1]);
    if constexpr (LOW) {
      lg[i] = pack16<F16>(left_over<F16>(a[0], og[i]), left_over<F16>(a[1], og[i] >> 16));
      lu[i] = pack16<F16>(left_over<F16>(b[0], ou[i]), left_over<F16>(b[1], ou[i] >> 16));
    }
  }
}

// The n (1 .. 8) first of eight 16-bit values to p.
__device__ __forceinline__ void store_part(uint16_t* p, u32x4 v, int n) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t w = v[e >> 1];
    if (e < n) p[e] = uint16_t(w >> (16 * (e & 1)));
  }
}

// The elementwise half, n = M N values in all (a multiple of 8).  Each thread
// reads its values before it writes them, so dG and dU may be any of the
// inputs' buffers.  dG and dU are rounded to the 16-bit type here, once: they are
// outputs of that type, and what the product takes; LOW: what the rounding left
// over goes to clg and clu.  Bound by memory, 5 x 2 (LOW: 7 x 2) bytes per value:
// 8192 x 5632 values take 68 us (6.8 TB/s; what was written last is partly still in
// the 256 MB cache), LOW 98 us.
template <bool F16, int ACT, bool LOW>
__global__ __launch_bounds__(kThreads) void glu_dgates_kernel(const uint16_t* g, const uint16_t* u, const uint16_t* dh,
                                                              uint16_t* dg, uint16_t* du, uint16_t* clg, uint16_t* clu,
                                                              int64_t n) {
  const int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 8;
  if (at >= n) return;
  u32x4 og, ou, lg, lu;
  dgates8<F16, ACT, LOW>(*reinterpret_cast<const u32x4*>(g + at), *reinterpret_cast<const u32x4*>(u + at),
                         *reinterpret_cast<const u32x4*>(dh + at), og, ou, lg, lu);
  *reinterpret_cast<u32x4*>(dg + at) = og;
  *reinterpret_cast<u32x4*>(du + at) = ou;
  if constexpr (LOW) {
    *reinterpret_cast<u32x4*>(clg + at) = lg;
    *reinterpret_cast<u32x4*>(clu + at) = lu;
  }
}

// The same for rows that are no multiple of 8 long: dG and dU also go to copies
// with rows of ld values, zeros behind the N-th, which the product reads (its
// 16-byte pieces need the alignment).
template <bool F16, int ACT, bool LOW>
__global__ __launch_bounds__(kThreads) void glu_dgates_ragged_kernel(const uint16_t* g, const uint16_t* u,
                                                                     const uint16_t* dh, uint16_t* dg, uint16_t* du,
                                                                     uint16_t* cg, uint16_t* cu, uint16_t* clg,
                                                                     uint16_t* clu, int64_t M, int N, int ld) {
  const int n = (blockIdx.y * kThreads + threadIdx.x) * 8, left = min(8, N - n);
  if (n >= ld) return;
  const bool whole = left == 8;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const int64_t at = m * N + n;
    u32x4 og, ou, lg, lu;
    dgates8<F16, ACT, LOW>(whole ? load8(g + at) : load_part(g + at, left),
                           whole ? load8(u + at) : load_part(u + at, left),
                           whole ? load8(dh + at) : load_part(dh + at, left), og, ou, lg, lu);
    *reinterpret_cast<u32x4*>(cg + m * ld + n) = og;  // dh is zero behind the row, so og and ou are
    *reinterpret_cast<u32x4*>(cu + m * ld + n) = ou;
    if constexpr (LOW) {
      *reinterpret_cast<u32x4*>(clg + m * ld + n) = lg;
      *reinterpret_cast<u32x4*>(clu + m * ld + n) = lu;
    }
    if (whole) {
      __builtin_memcpy(dg + at, &og, 16);
      __builtin_memcpy(du + at, &ou, 16);
    } else {
      store_part(dg + at, og, left);
      store_part(du + at, ou, left);
    }
  }
}

// dX from the splits' partial sums: four threads take every fourth split of four
// values, then their sums are added in order (one thread over all splits took
// 9 us for 24 x 2048 values and 32 splits: one load after the other).  Bound by
// the latency of splits / 4 loads, in a fixed order, so results repeat bit by bit.
template <bool F16>
__global__ __launch_bounds__(kThreads) void glu_join_kernel(const float* part, uint16_t* dx, int64_t n, int splits) {
  __shared__ f32x4 sums[4][kThreads / 4];
  const int i = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int64_t at = (int64_t(blockIdx.x) * 64 + i) * 4;  // n is a multiple of 32
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (at < n)
#pragma unroll 4
    for (int s = g; s < splits; s += 4) v += *reinterpret_cast<const f32x4*>(part + s * n + at);
  sums[g][i] = v;
  __syncthreads();
  if (g || at >= n) return;
  v = ((sums[0][i] + sums[1][i]) + sums[2][i]) + sums[3][i];
  *reinterpret_cast<u32x2*>(dx + at) = u32x2{pack16<F16>(v[0], v[1]), pack16<F16>(v[2], v[3])};
}

}  // namespace

// Which tile and how many splits of the depth: the cut with the smallest
// estimate.  Us per stage of 32 rows, by tile and by the workgroups on a compute
// unit (as many as their LDS allows), what a round of the chip adds, and what the
// join costs (its launch and its bytes), fitted to 5191 timings (W4A16, Q4K, Q8_0
// and dense; 1 to 4096 tokens of 64 x 256 to 5632 x 2048): on average 1 % and at
// most 12 % over the best cut of each size.  W4A16, 5632 x 2048: 512 tokens 57.9
// with 128 x 128 and 8 splits against 63.5 with 256 x 256 and 16, 2048 tokens 140
// with 256 x 256 and 4 against 177 with 128 x 128 and 2.  The same cut serves the
// form with low parts, whose best cuts are the same or next to it: W4A16, 5632 x
// 2048, the rule's is the best measured one at 1, 24, 391, 512, 2048 and 8192 tokens
// and 3 to 4 % over it at 64 and 128; over 36 sizes of four formats 2 % on average,
// at most 19 % (Q8_0, 1024 x 768, 2048 tokens: 44.5 against 37.5).  Past the fitted
// sizes, 14336 x 4096 (W4A16, Q4K) and 8192 x 2816 (Q6K) with 1 to 4096 tokens, the cut
// is the best measured one at all 24 sizes; with low parts 4 % over it on average, at
// most 23 % (Q6K, 1024 tokens: 330 against 268 with 128 x 128, as the large tile spills).
GluBwdPlan glu_backward_plan(int64_t N, int64_t K, int64_t M, bool wide) {
  struct Tile {
    int k, m, units;  // columns, tokens; workgroups that share a unit
    double stage[3], round;
  };
  constexpr Tile kTiles[3] = {
      {128, 64, 3, {0.25, 0.37, 0.69}, 0.6}, {128, 128, 2, {0.33, 0.52}, 1.5}, {256, 256, 1, {0.68}, 5.4}};
  GluBwdPlan best{};
  const int64_t stages = 2 * ((N + 31) / 32);
  double best_us = 0;
  for (int64_t cut : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
    if (cut > 1 && stages / cut < 4) break;
    const int64_t steps = ((stages + cut - 1) / cut + 3) / 4 * 4;
    const int64_t splits = (stages + steps - 1) / steps;  // no empty split
    for (int t = 0; t < 3; ++t) {
      const Tile& c = kTiles[t];
      const int64_t tiles = ((K + c.k - 1) / c.k) * ((M + c.m - 1) / c.m), groups = tiles * splits;
      const int64_t full = groups / (256 * c.units), rest = (groups - full * 256 * c.units + 255) / 256;
      double us = double(full) * (c.stage[c.units - 1] * double(steps) + c.round);
      if (rest) us += c.stage[rest - 1] * double(steps) + c.round;
      if (splits > 1) us += 2.0 + double(splits) * double(M) * double(K) * 8e-6 * 0.13;
      if (best.tiles && us >= best_us) continue;
      best_us = us;
      best = GluBwdPlan{t, int(splits), int(steps), 0, tiles, splits > 1 ? splits * M * K * 4 : 0, 0, 0};
    }
  }
  best.ld = int((N + 7) / 8 * 8);
  const int64_t copy = M * best.ld * 2;  // a multiple of 16
  if (N % 8) best.copy_bytes = copy;
  if (wide) best.low_bytes = copy;
  return best;
}

hipError_t launch_glu_fwd(int fmt, int64_t N, int64_t K, int64_t M, const uint8_t* Wg, const uint8_t* Wu,
                          const uint16_t* X, bool f16, int act, uint16_t* H, uint16_t* G, uint16_t* U, hipStream_t s) {
  const Planes pl = planes_of(fmt, N, K);
  const GluFwdArgs p{mat_of(Wg, pl), mat_of(Wu, pl), X, H, G, U, int(M), int(N), int(K), act};
  switch (fmt) {
    case QMV_W4A16_G64: case QMV_Q4K: case QMV_DENSE_BF16: return launch_glu_fwd_a(fmt, f16, p, s);
    case QMV_Q8_0: case QMV_Q6K: case QMV_I8_ROW: return launch_glu_fwd_b(fmt, f16, p, s);
    default: return launch_glu_fwd_c(fmt, f16, p, s);
  }
}

hipError_t launch_glu_bwd(int fmt, int64_t N, int64_t K, int64_t M, const uint8_t* Wg, const uint8_t* Wu,
                          const uint16_t* G, const uint16_t* U, const uint16_t* dH, bool f16, int act,
                          const GluBwdPlan& plan, uint16_t* dG, uint16_t* dU, uint16_t* dX, uint8_t* ws, hipStream_t s) {
  const Planes pl = planes_of(fmt, N, K);
  const int64_t mn = M * N, mk = M * K;
  uint16_t *cg = dG, *cu = dU, *clg = nullptr, *clu = nullptr;
  uint8_t* at = ws + plan.part_bytes;
  if (plan.copy_bytes) {
    cg = reinterpret_cast<uint16_t*>(at);
    cu = reinterpret_cast<uint16_t*>(at + plan.copy_bytes);
    at += 2 * plan.copy_bytes;
  }
  if (plan.low_bytes) {
    clg = reinterpret_cast<uint16_t*>(at);
    clu = reinterpret_cast<uint16_t*>(at + plan.low_bytes);
  }
  auto gates = [&]<bool F16, int ACT, bool LOW>() {
    if (plan.copy_bytes) {
      const dim3 grid(unsigned(std::min<int64_t>(M, 1 << 20)), unsigned((plan.ld / 8 + kThreads - 1) / kThreads));
      hipLaunchKernelGGL((glu_dgates_ragged_kernel<F16, ACT, LOW>), grid, dim3(kThreads), 0, s, G, U, dH, dG, dU, cg,
                         cu, clg, clu, M, int(N), plan.ld);
    } else {
      const dim3 grid(unsigned((mn + 8 * kThreads - 1) / (8 * kThreads)));
      hipLaunchKernelGGL((glu_dgates_kernel<F16, ACT, LOW>), grid, dim3(kThreads), 0, s, G, U, dH, dG, dU, clg, clu,
                         mn);
    }
  };
  auto by_act = [&]<bool F16, bool LOW>() {
    if (act == QMV_ACT_SILU) gates.template operator()<F16, QMV_ACT_SILU, LOW>();
    else if (act == QMV_ACT_GELU_TANH) gates.template operator()<F16, QMV_ACT_GELU_TANH, LOW>();
    else gates.template operator()<F16, QMV_ACT_GELU, LOW>();
  };
  if (plan.low_bytes) f16 ? by_act.template operator()<true, true>() : by_act.template operator()<false, true>();
  else f16 ? by_act.template operator()<true, false>() : by_act.template operator()<false, false>();
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* part = plan.splits > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  const GluBwdArgs p{mat_of(Wg, pl), mat_of(Wu, pl), cg, cu, clg, clu, dX, part, int(M), int(N), int(K), plan.ld,
                     plan.steps};
  switch (fmt) {
    case QMV_W4A16_G64: case QMV_Q4K: case QMV_DENSE_BF16: e = launch_glu_bwd_a(fmt, f16, p, plan, s); break;
    case QMV_Q8_0: case QMV_Q6K: case QMV_I8_ROW: e = launch_glu_bwd_b(fmt, f16, p, plan, s); break;
    default: e = launch_glu_bwd_c(fmt, f16, p, plan, s); break;
  }
  if (e != hipSuccess || !part) return e;
  const dim3 jg(static_cast<unsigned>((mk + 255) / 256));
  if (f16) hipLaunchKernelGGL(glu_join_kernel<true>, jg, dim3(kThreads), 0, s, part, dX, mk, plan.splits);
  else hipLaunchKernelGGL(glu_join_kernel<false>, jg, dim3(kThreads), 0, s, part, dX, mk, plan.splits);
  return hipGetLastError();
}

}  // namespace qmv
