// The gated products of many tokens, H = act(X Wg^T) * (X Wu^T), on the matrix cores.
#pragma once

#include "gemm16.h"

namespace qmv {

struct GluFwdArgs {
  Mat wg, wu;
  const uint16_t* x;
  uint16_t *h, *g, *u;  // g, u may be null (both)
  int M, N, K, act;
  int vec;              // rows of h, g, u may be written 8 bytes at a time
};

namespace {

// RB, TB: 32-row blocks of weights (half gate, half up) and of tokens per wave;
// WR x WT waves.  A step takes 64 of K.
template <int FMT, bool F16, int RB, int TB, int WR, int WT>
__global__ __launch_bounds__(64 * WR * WT) void glu_fwd_kernel(const GluFwdArgs p) {
  constexpr int NT = 64 * WR * WT;
  constexpr int BR = 32 * RB * WR, BN = BR / 2, BM = 32 * TB * WT;
  constexpr int UPT = 2 * BR / NT;      // weight units per thread and step
  constexpr int XPT = BM * 8 / NT;      // 16-byte token pieces per thread and step
  static_assert(UPT * NT == 2 * BR && XPT * NT == BM * 8 && RB % 2 == 0);

  __shared__ u32x4 As[2][BR * 8];
  __shared__ u32x4 Xs[2][BM * 8];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WT, wt = wave % WT;
  const int n0 = blockIdx.x * BN, m0 = blockIdx.y * BM;
  const int K = p.K, U = K >> 5, ns = (K + 63) >> 6;

  // this thread's weight units: unit uu (0, 1) of LDS row ra, which is a gate or an up row
  struct Set {
    UnitRaw<FMT> w[UPT];
    u32x4 x[XPT];
  };
  auto load = [&](Set& s, int step) {
#pragma unroll
    for (int j = 0; j < UPT; ++j) {
      const int id = j * NT + tid, ra = id % BR, uu = id / BR;
      const int q = ra % (32 * RB);
      const bool up = q >= 16 * RB;
      const int n = min(n0 + (ra / (32 * RB)) * 16 * RB + q % (16 * RB), p.N - 1);
      s.w[j] = load_unit<FMT>(up ? p.wu : p.wg, n, min(2 * step + uu, U - 1), K);
    }
#pragma unroll
    for (int j = 0; j < XPT; ++j) {
      const int id = j * NT + tid, r = id >> 3, c = id & 7;
      const int m = min(m0 + r, p.M - 1), k = min(64 * step + 8 * c, K - 8);
      s.x[j] = *reinterpret_cast<const u32x4*>(p.x + int64_t(m) * K + k);
    }
  };
  auto stage = [&](const Set& s, int step, int buf) {
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < XPT; ++j) {
      const int id = j * NT + tid, r = id >> 3, c = id & 7;
      Xs[buf][tile_at(r, c)] = 64 * step + 8 * c < K ? s.x[j] : zero;
    }
#pragma unroll
    for (int j = 0; j < UPT; ++j) {
      const int id = j * NT + tid, ra = id % BR, uu = id / BR;
      const int u = 2 * step + uu;
      const Affine f = affine_of<FMT>(s.w[j].m, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4 v = unit_piece<FMT, F16>(s.w[j], f, i);
        As[buf][tile_at(ra, 4 * uu + i)] = u < U ? v : zero;
      }
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
      for (int i = 0; i < RB; ++i) a[i] = As[buf][tile_at((wr * RB + i) * 32 + fr, 2 * s + fh)];
#pragma unroll
      for (int i = 0; i < TB; ++i) b[i] = Xs[buf][tile_at((wt * TB + i) * 32 + fr, 2 * s + fh)];
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = mfma32<F16>(a[i], b[j], acc[i][j]);
    }
  };

  Set s0, s1;
  load(s0, 0);
  load(s1, min(1, ns - 1));
  stage(s0, 0, 0);
  lds_barrier16();
  int st = 0;
  for (; st + 1 < ns; st += 2) {
    load(s0, min(st + 2, ns - 1));
    stage(s1, st + 1, 1);
    products(0);
    lds_barrier16();
    load(s1, min(st + 3, ns - 1));
    stage(s0, min(st + 2, ns - 1), 0);
    products(1);
    lds_barrier16();
  }
  if (st < ns) products(0);

  // C fragment: lane holds rows n = 8 q + 4 fh + e (q, e in 0..3) of token lane % 32
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const int m = m0 + (wt * TB + j) * 32 + fr;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < RB / 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + (wr * (RB / 2) + i) * 32 + 8 * q + 4 * fh;
        float g[4], u[4], h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = acc[i][j][4 * q + e];
          u[e] = acc[i + RB / 2][j][4 * q + e];
          h[e] = act_value(p.act, g[e]) * u[e];
        }
        auto put = [&](uint16_t* y, const float (&v)[4]) {
          uint16_t* d = y + int64_t(m) * p.N + n;
          const uint32_t lo = pack16<F16>(v[0], v[1]), hi = pack16<F16>(v[2], v[3]);
          if (p.vec && n + 3 < p.N) {
            *reinterpret_cast<u32x2*>(d) = u32x2{lo, hi};
          } else {
            if (n < p.N) d[0] = uint16_t(lo);
            if (n + 1 < p.N) d[1] = uint16_t(lo >> 16);
            if (n + 2 < p.N) d[2] = uint16_t(hi);
            if (n + 3 < p.N) d[3] = uint16_t(hi >> 16);
          }
        };
        put(p.h, h);
        if (p.g) {
          put(p.g, g);
          put(p.u, u);
        }
      }
  }
}

// Few tokens: a weight stream.  A workgroup owns 16 gate and the same 16 up
// rows; its W waves split K in steps of 128 (wave w takes steps w, w + W, ...).
// Lane group g (16 lanes) of a fragment holds one 32-k unit, word s of it being
// k = 32 g + 8 s .. + 7 of MFMA s; the token operand follows the same order
// straight from global memory (no two waves share a step, so LDS would only be
// a detour).  The partial tiles meet in LDS and are added in wave order.
template <int FMT, bool F16, int FM, int W>
__global__ __launch_bounds__(64 * W) void glu_fwd_few_kernel(const GluFwdArgs p) {
  __shared__ f32x4 red[W][2 * FM][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g4 = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * FM;
  const int K = p.K, U = K >> 5, nk = (K + 127) >> 7;
  const int n = min(n0 + fr, p.N - 1);

  struct Set {
    UnitRaw<FMT> g, u;
    u32x4 x[FM][4];
  };
  auto load = [&](Set& s, int step) {
    const int u = min(4 * step + g4, U - 1);
    s.g = load_unit<FMT>(p.wg, n, u, K);
    s.u = load_unit<FMT>(p.wu, n, u, K);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int m = min(m0 + 16 * j + fr, p.M - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s.x[j][i] = *reinterpret_cast<const u32x4*>(p.x + int64_t(m) * K + 32 * u + 8 * i);
    }
  };
  f32x4 acc[2][FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) acc[0][j] = acc[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Set& s, int step) {
    const int u = 4 * step + g4;
    const bool in = u < U;
    const u32x4 zero = {0, 0, 0, 0};
    const Affine fg = affine_of<FMT>(s.g.m, min(u, U - 1)), fu = affine_of<FMT>(s.u.m, min(u, U - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 vg = unit_piece<FMT, F16>(s.g, fg, i), vu = unit_piece<FMT, F16>(s.u, fu, i);
      const u32x4 ag = in ? vg : zero, au = in ? vu : zero;
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const u32x4 b = in ? s.x[j][i] : zero;
        acc[0][j] = mfma16<F16>(ag, b, acc[0][j]);
        acc[1][j] = mfma16<F16>(au, b, acc[1][j]);
      }
    }
  };
  Set s0, s1;
  load(s0, wave);
  load(s1, wave + W);
  for (int st = wave; st < nk; st += 2 * W) {
    use(s0, st);
    load(s0, st + 2 * W);
    use(s1, st + W);  // all zeros past the last step
    load(s1, st + 3 * W);
  }
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    red[wave][2 * j][lane] = acc[0][j];
    red[wave][2 * j + 1][lane] = acc[1][j];
  }
  lds_barrier16();
  // C fragment: lane holds rows n0 + 4 g4 + e of token fr
  for (int j = wave; j < FM; j += W) {
    f32x4 g = red[0][2 * j][lane], u = red[0][2 * j + 1][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      g += red[w][2 * j][lane];
      u += red[w][2 * j + 1][lane];
    }
    const int m = m0 + 16 * j + fr;
    if (m < p.M) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int nn = n0 + 4 * g4 + e;
        if (nn < p.N) {
          const int64_t at = int64_t(m) * p.N + nn;
          p.h[at] = uint16_t(pack16<F16>(act_value(p.act, g[e]) * u[e], 0.f));
          if (p.g) {
            p.g[at] = uint16_t(pack16<F16>(g[e], 0.f));
            p.u[at] = uint16_t(pack16<F16>(u[e], 0.f));
          }
        }
      }
    }
  }
}

template <int FMT, bool F16>
hipError_t glu_fwd_go(const GluFwdArgs& p, hipStream_t s) {
  if (p.M <= 64) {
    const dim3 grid((p.N + 15) / 16);
    if (p.M <= 16)
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 1, 4>), grid, dim3(256), 0, s, p);
    else if (p.M <= 32)
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 2, 4>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 4, 4>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
  }
  const int64_t big = int64_t((p.N + 127) / 128) * ((p.M + 255) / 256);
  if (big >= 256) {
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, 4, 2, 2, 4>), dim3((p.N + 127) / 128, (p.M + 255) / 256), dim3(512), 0,
                       s, p);
  } else {
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, 2, 2, 2, 2>), dim3((p.N + 63) / 64, (p.M + 127) / 128), dim3(256), 0, s,
                       p);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace qmv
