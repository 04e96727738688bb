// Backward pass of the gated products: dX = dG Wg + dU Wu, on the matrix cores.
#pragma once

#include "gemm16.h"

namespace qmv {

struct GluBwdArgs {
  Mat wg, wu;
  const uint16_t *dg, *du;
  uint16_t* dx;
  float* part;      // [splits][M][K] partial sums, or null: one split, dx written
  int M, N, K;
  int steps;        // contraction steps per split
};

namespace {

// Rows of the tile are BR columns k of dX, its depth runs over n: first the
// gate rows, then the up rows, 64 per step.
template <int FMT, bool F16, int RB, int TB, int WR, int WT>
__global__ __launch_bounds__(64 * WR * WT) void glu_bwd_kernel(const GluBwdArgs p) {
  constexpr int NT = 64 * WR * WT;
  constexpr int BR = 32 * RB * WR, BM = 32 * TB * WT;
  constexpr int BPT = BR / NT > 0 ? BR / NT : 1;  // 8 x 8 weight blocks per thread and step
  constexpr int XPT = BM * 8 / NT;
  constexpr bool SOME = BR < NT;                   // only the first BR threads hold a block
  static_assert((SOME || BPT * NT == BR) && XPT * NT == BM * 8);

  __shared__ u32x4 As[2][BR * 8];
  __shared__ u32x4 Xs[2][BM * 8];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WT, wt = wave % WT;
  const int k0 = blockIdx.x * BR, m0 = blockIdx.y * BM;
  const int N = p.N, K = p.K;
  const int half = (N + 63) >> 6;  // steps per matrix
  const int first = blockIdx.z * p.steps, ns = min(p.steps, 2 * half - first);

  struct Set {
    WordRaw<FMT> w[BPT][8];
    u32x4 x[XPT];
  };
  constexpr int KG = BR / 8;  // groups of 8 columns
  auto load = [&](Set& s, int step) {
    const bool up = step >= half;
    const int nb = 64 * (up ? step - half : step);
    const Mat wn = from_row<FMT>(up ? p.wu : p.wg, nb, K);
    const uint16_t* d = up ? p.du : p.dg;
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      const int id = (j * NT + tid) % BR, kg = id % KG, ng = id / KG;
      const int kw = min((k0 >> 3) + kg, (K >> 3) - 1);
#pragma unroll
      for (int e = 0; e < 8; ++e) s.w[j][e] = load_word<FMT>(wn, min(nb + 8 * ng + e, N - 1) - nb, kw >> 2, kw & 3, K);
    }
#pragma unroll
    for (int j = 0; j < XPT; ++j) {
      const int id = j * NT + tid, r = id >> 3, c = id & 7;
      const int m = min(m0 + r, p.M - 1), n = nb + 8 * c;
      const uint16_t* q = d + int64_t(m) * N + n;
      if (n + 8 <= N) s.x[j] = load8(q);
      else s.x[j] = load_part(q, N - n);  // zeros where n >= N
    }
  };
  auto stage = [&](const Set& s, int step, int buf) {
    const bool up = step >= half;
    const int nb = 64 * (up ? step - half : step);
#pragma unroll
    for (int j = 0; j < XPT; ++j) {
      const int id = j * NT + tid, r = id >> 3, c = id & 7;
      Xs[buf][tile_at(r, c)] = s.x[j];
    }
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      if (SOME && tid >= BR) break;
      const int id = (j * NT + tid) % BR, kg = id % KG, ng = id / KG;
      const int kw = min((k0 >> 3) + kg, (K >> 3) - 1);
      u32x4 o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a[8], b[8];
        word_values<FMT>(s.w[j][2 * e], kw >> 2, kw & 3, a);
        word_values<FMT>(s.w[j][2 * e + 1], kw >> 2, kw & 3, b);
        const bool ina = nb + 8 * ng + 2 * e < N, inb = nb + 8 * ng + 2 * e + 1 < N;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k][e] = pack16<F16>(ina ? a[k] : 0.0f, inb ? b[k] : 0.0f);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) As[buf][tile_at_t(8 * kg + k, ng)] = o[k];
    }
  };

  f32x16 acc[RB][TB];
#pragma unroll
  for (int a = 0; a < RB; ++a)
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.0f;

  const int fr = lane & 31, fh = lane >> 5;
  auto products = [&](int buf) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 a[RB], b[TB];
#pragma unroll
      for (int i = 0; i < RB; ++i) a[i] = As[buf][tile_at_t((wr * RB + i) * 32 + fr, 2 * s + fh)];
#pragma unroll
      for (int i = 0; i < TB; ++i) b[i] = Xs[buf][tile_at((wt * TB + i) * 32 + fr, 2 * s + fh)];
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = mfma32<F16>(a[i], b[j], acc[i][j]);
    }
  };

  Set s0, s1;
  const int last = first + ns - 1;
  load(s0, first);
  load(s1, min(first + 1, last));
  stage(s0, first, 0);
  lds_barrier16();
  int st = first;
  for (; st < last; st += 2) {
    load(s0, min(st + 2, last));
    stage(s1, st + 1, 1);
    products(0);
    lds_barrier16();
    load(s1, min(st + 3, last));
    stage(s0, min(st + 2, last), 0);
    products(1);
    lds_barrier16();
  }
  if (st == last) products(0);

#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const int m = m0 + (wt * TB + j) * 32 + fr;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = k0 + (wr * RB + i) * 32 + 8 * q + 4 * fh;
        if (k >= K) continue;  // K is a multiple of 32: all four or none
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
        const int64_t at = int64_t(m) * K + k;
        if (p.part)
          *reinterpret_cast<f32x4*>(p.part + int64_t(blockIdx.z) * p.M * K + at) = v;
        else
          *reinterpret_cast<u32x2*>(p.dx + at) = u32x2{pack16<F16>(v[0], v[1]), pack16<F16>(v[2], v[3])};
      }
  }
}

template <int FMT, bool F16>
hipError_t glu_bwd_go(const GluBwdArgs& p, int splits, hipStream_t s) {
  const dim3 grid((p.K + 127) / 128, (p.M + 127) / 128, splits);
  const int64_t big = int64_t((p.K + 255) / 256) * ((p.M + 255) / 256);
  if (p.M <= 32)
    hipLaunchKernelGGL((glu_bwd_kernel<FMT, F16, 1, 1, 4, 1>), dim3(grid.x, (p.M + 31) / 32, splits), dim3(256), 0, s, p);
  else if (big >= 256)
    hipLaunchKernelGGL((glu_bwd_kernel<FMT, F16, 4, 2, 2, 4>), dim3((p.K + 255) / 256, (p.M + 255) / 256, splits),
                       dim3(512), 0, s, p);
  else
    hipLaunchKernelGGL((glu_bwd_kernel<FMT, F16, 2, 2, 2, 2>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace qmv
