// Gated products of many tokens: dispatch, the elementwise half of the backward
// pass and the sum of its split partials.
#include <algorithm>

#include "glu_bwd.h"
#include "glu_fwd.h"

namespace qmv {

hipError_t launch_glu_fwd_a(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s);
hipError_t launch_glu_fwd_b(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s);
hipError_t launch_glu_fwd_c(int fmt, bool f16, const GluFwdArgs& p, hipStream_t s);
hipError_t launch_glu_bwd_a(int fmt, bool f16, const GluBwdArgs& p, int splits, hipStream_t s);
hipError_t launch_glu_bwd_b(int fmt, bool f16, const GluBwdArgs& p, int splits, hipStream_t s);
hipError_t launch_glu_bwd_c(int fmt, bool f16, const GluBwdArgs& p, int splits, hipStream_t s);

namespace {

constexpr int kThreads = 256;

// dG = dH U act'(G), dU = dH act(G), eight values per thread.  Each thread
// reads its values before it writes them, so dG and dU may be any of the
// inputs' buffers.  n values in all.
template <bool F16, int ACT>
__global__ __launch_bounds__(kThreads) void glu_dgates_kernel(const uint16_t* g, const uint16_t* u, const uint16_t* dh,
                                                              uint16_t* dg, uint16_t* du, int64_t n) {
  const int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 8;
  if (at >= n) return;
  const bool whole = at + 8 <= n;
  const int left = int(min(n - at, int64_t(8)));
  const u32x4 gv = whole ? *reinterpret_cast<const u32x4*>(g + at) : load_part(g + at, left);
  const u32x4 uv = whole ? *reinterpret_cast<const u32x4*>(u + at) : load_part(u + at, left);
  const u32x4 hv = whole ? *reinterpret_cast<const u32x4*>(dh + at) : load_part(dh + at, left);
  u32x4 og, ou;
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
  }
  if (whole) {
    *reinterpret_cast<u32x4*>(dg + at) = og;
    *reinterpret_cast<u32x4*>(du + at) = ou;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) {
        dg[at + e] = uint16_t(og[e >> 1] >> (16 * (e & 1)));
        du[at + e] = uint16_t(ou[e >> 1] >> (16 * (e & 1)));
      }
  }
}

// dX from the splits' partial sums, added in split order.
template <bool F16>
__global__ __launch_bounds__(kThreads) void glu_join_kernel(const float* part, uint16_t* dx, int64_t n, int splits) {
  const int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 4;  // n is a multiple of 32
  if (at >= n) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(part + at);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(part + s * n + at);
  *reinterpret_cast<u32x2*>(dx + at) = u32x2{pack16<F16>(v[0], v[1]), pack16<F16>(v[2], v[3])};
}

}  // namespace

int glu_backward_splits(int64_t N, int64_t K, int64_t M) {
  const int64_t bm = M <= 32 ? 32 : 128;
  const int64_t tiles = ((K + 127) / 128) * ((M + bm - 1) / bm);
  const int64_t steps = 2 * ((N + 63) / 64);
  return int(std::max<int64_t>(1, std::min<int64_t>({512 / tiles, steps / 4, 32})));
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
                          const uint16_t* G, const uint16_t* U, const uint16_t* dH, bool f16, int act, uint16_t* dG,
                          uint16_t* dU, uint16_t* dX, float* ws, int splits, hipStream_t s) {
  const Planes pl = planes_of(fmt, N, K);
  const int64_t mn = M * N, mk = M * K;
  const dim3 eg(static_cast<unsigned>((mn + 8 * kThreads - 1) / (8 * kThreads)));
  auto gates = [&]<int ACT>() {
    if (f16) hipLaunchKernelGGL((glu_dgates_kernel<true, ACT>), eg, dim3(kThreads), 0, s, G, U, dH, dG, dU, mn);
    else hipLaunchKernelGGL((glu_dgates_kernel<false, ACT>), eg, dim3(kThreads), 0, s, G, U, dH, dG, dU, mn);
  };
  if (act == QMV_ACT_SILU) gates.template operator()<QMV_ACT_SILU>();
  else if (act == QMV_ACT_GELU_TANH) gates.template operator()<QMV_ACT_GELU_TANH>();
  else gates.template operator()<QMV_ACT_GELU>();
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int steps = int(2 * ((N + 63) / 64));
  const int per = (steps + splits - 1) / splits;
  splits = (steps + per - 1) / per;  // no empty split
  const GluBwdArgs p{mat_of(Wg, pl), mat_of(Wu, pl), dG, dU, dX, splits > 1 ? ws : nullptr, int(M), int(N), int(K), per};
  switch (fmt) {
    case QMV_W4A16_G64: case QMV_Q4K: case QMV_DENSE_BF16: e = launch_glu_bwd_a(fmt, f16, p, splits, s); break;
    case QMV_Q8_0: case QMV_Q6K: case QMV_I8_ROW: e = launch_glu_bwd_b(fmt, f16, p, splits, s); break;
    default: e = launch_glu_bwd_c(fmt, f16, p, splits, s); break;
  }
  if (e != hipSuccess || splits == 1) return e;
  const dim3 jg(static_cast<unsigned>((mk + 4 * kThreads - 1) / (4 * kThreads)));
  if (f16) hipLaunchKernelGGL(glu_join_kernel<true>, jg, dim3(kThreads), 0, s, ws, dX, mk, splits);
  else hipLaunchKernelGGL(glu_join_kernel<false>, jg, dim3(kThreads), 0, s, ws, dX, mk, splits);
  return hipGetLastError();
}

}  // namespace qmv
