// The gated products of many tokens, H = act(X Wg^T) * (X Wu^T), on the matrix cores.
#pragma once

#include "gemm16.h"

namespace qmv {

struct GluFwdArgs {
  Mat wg, wu;
  const uint16_t* x;
  uint16_t *h, *g, *u;  // g, u may be null (both)
  int M, N, K, act;
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

  // let the tiles' addresses escape: otherwise the compiler knows that no asm
  // statement can touch them and moves LDS reads across the fences below
  asm volatile("" ::"v"(&As[0][0]), "v"(&Xs[0][0]) : "memory");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WT, wt = wave % WT;
  const TileId id0 = tile_of_block(p.N, BN, p.M, BM);
  const int n0 = id0.x * BN, m0 = id0.y * BM;
  const int K = p.K, U = K >> 5, last = ((K + 63) >> 6) - 1;

  // Thread tid stages units of weight row n0 + tid % BN: of the gate or the up
  // matrix and of which half of the step goes by wave, so that the addresses
  // are scalar bases and one lane offset per plane.
  const uint32_t wrow = min(n0 + tid % BN, p.N - 1) - n0;
  const int wq = wave / (BN / 64);                       // gate / up and half of this wave's first unit
  const Mat wg = from_row<FMT>(p.wg, n0, K), wu = from_row<FMT>(p.wu, n0, K);
  constexpr int QPW = (2 * BR / 64) / UPT / (BN / 64);   // (matrix, half) pairs that the waves cover at once
  const int arow = ((tid % BN) / (16 * RB)) * 32 * RB + (tid % BN) % (16 * RB);
  // token pieces: row tid / 8 + j * NT / 8, piece tid % 8
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x + int64_t(m0) * K);
  uint32_t xo[XPT];
#pragma unroll
  for (int j = 0; j < XPT; ++j) xo[j] = uint32_t(min(m0 + j * (NT / 8) + (tid >> 3), p.M - 1) - m0) * uint32_t(2 * K);

  struct Set {
    UnitRaw<FMT> w[UPT];
    u32x4 x[XPT];
  };
  auto load = [&](Set& s, int step) {
    const int whole = 2 * step + 1 < U;  // else half a step: its first half twice
#pragma unroll
    for (int j = 0; j < UPT; ++j) {
      const int q = wq + j * QPW, uu = q >> 1;
      s.w[j] = load_unit<FMT, false>(q & 1 ? wu : wg, wrow, 2 * step + (whole ? uu : 0), K);
    }
    const uint32_t c = 16 * (tid & (whole ? 7 : 3));
#pragma unroll
    for (int j = 0; j < XPT; ++j) s.x[j] = load_at<u32x4>(xb + 128 * int64_t(step), xo[j] + c);
  };
  // part i (0..3) of a step's staging: word i of the thread's units, and its
  // share of the token pieces
  auto stage = [&](const Set& s, int step, int buf, int i) {
#pragma unroll
    for (int j = 0; j < XPT; ++j) {
      if (j * 4 / XPT != i) continue;
      const int id = j * NT + tid;
      Xs[buf][tile_at(id >> 3, id & 7)] = s.x[j];
    }
#pragma unroll
    for (int j = 0; j < UPT; ++j) {
      const int q = wq + j * QPW, uu = q >> 1;
      As[buf][tile_at(arow + (q & 1) * 16 * RB, 4 * uu + i)] =
          unit_piece<FMT, F16>(s.w[j], affine_of<FMT>(s.w[j].m, 2 * step + uu), i);
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
  struct Frag {
    u32x4 a[RB], b[TB];
  };
  auto read = [&](Frag& f, int buf, int s) {
#pragma unroll
    for (int i = 0; i < RB; ++i) f.a[i] = As[buf][tile_at((wr * RB + i) * 32 + fr, 2 * s + fh)];
#pragma unroll
    for (int i = 0; i < TB; ++i) f.b[i] = Xs[buf][tile_at((wt * TB + i) * 32 + fr, 2 * s + fh)];
  };
  auto mul = [&](const Frag& f) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j) acc[i][j] = mfma32<F16>(f.a[i], f.b[j], acc[i][j]);
  };
  // One step: products of buffer `buf` while the next step (already in `next`)
  // is decoded into the other buffer and the one after it is loaded into `then`.
  // The fences keep the loads at the top and the LDS traffic spread.
  auto fence = [] {
    asm volatile("" ::: "memory");
#ifndef VAR_NOSB
    __builtin_amdgcn_sched_barrier(0);
#endif
  };
  auto step = [&](int st, int buf, Set& then, const Set& next) {
    Frag f0, f1;
    read(f0, buf, 0);
    load(then, min(st + 2, last));
    fence();
    read(f1, buf, 1);
    stage(next, st + 1, buf ^ 1, 0);
    mul(f0);
    fence();
    read(f0, buf, 2);
    stage(next, st + 1, buf ^ 1, 1);
    mul(f1);
    fence();
    read(f1, buf, 3);
    stage(next, st + 1, buf ^ 1, 2);
    mul(f0);
    fence();
    stage(next, st + 1, buf ^ 1, 3);
    mul(f1);
    lds_barrier16();
  };

  // whole steps, then half a step (K is a multiple of 32): units and pieces
  // past K are loaded from clamped addresses and never multiplied
  const int nf = K >> 6;
  Set s0, s1;
  load(s0, 0);
  load(s1, min(1, last));
#pragma unroll
  for (int i = 0; i < 4; ++i) stage(s0, 0, 0, i);
  lds_barrier16();
  int st = 0;
  for (; st + 1 < nf; st += 2) {
    step(st, 0, s0, s1);
    step(st + 1, 1, s1, s0);
  }
  if (st < nf) {
    step(st, 0, s0, s1);
    ++st;
  }
  if (K & 32) {
    Frag f0, f1;
    read(f0, st & 1, 0);
    read(f1, st & 1, 1);
    mul(f0);
    mul(f1);
  }

  // C fragment: lane holds rows n = 8 q + 4 fh + e (q, e in 0..3) of token
  // lane % 32.  Each output goes through the wave's own part of LDS (the tiles
  // are done with), so that rows of up to 128 bytes leave whole.
  lds_barrier16();
  constexpr int HB = RB / 2;                       // 32-row blocks of outputs
  u32x4* mine = &As[0][0] + wave * (32 * 8);       // 32 tokens x 64 values
  const int nw = n0 + wr * HB * 32;
  auto put = [&](uint16_t* y, int j, auto value) {
#pragma unroll
    for (int i = 0; i < HB; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = value(i, 4 * q + e);
        reinterpret_cast<u32x2*>(mine + tile_at(fr, 4 * i + q))[fh] = u32x2{pack16<F16>(v[0], v[1]), pack16<F16>(v[2], v[3])};
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // written and read by this wave only
    constexpr int PPR = 4 * HB;  // 16-byte pieces per row
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 64 / PPR) {
      const int r = r0 + lane / PPR, c = lane % PPR;
      const u32x4 v = mine[tile_at(r, c)];
      const int m = m0 + (wt * TB + j) * 32 + r, n = nw + 8 * c;
      if (m < p.M) {
        uint16_t* d = y + int64_t(m) * p.N + n;
        if (n + 8 <= p.N) {
          __builtin_memcpy(d, &v, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t w = v[e >> 1];
            if (n + e < p.N) d[e] = uint16_t(w >> (16 * (e & 1)));
          }
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  auto out = [&]<int ACT>() {
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      put(p.h, j, [&](int i, int e) { return act_value<ACT>(acc[i][j][e]) * acc[i + HB][j][e]; });
      if (p.g) {
        put(p.g, j, [&](int i, int e) { return acc[i][j][e]; });
        put(p.u, j, [&](int i, int e) { return acc[i + HB][j][e]; });
      }
    }
  };
  if (p.act == QMV_ACT_SILU) out.template operator()<QMV_ACT_SILU>();
  else if (p.act == QMV_ACT_GELU_TANH) out.template operator()<QMV_ACT_GELU_TANH>();
  else out.template operator()<QMV_ACT_GELU>();
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
  const uint32_t row = min(n0 + fr, p.N - 1) - n0;
  const Mat wg = from_row<FMT>(p.wg, n0, K), wu = from_row<FMT>(p.wu, n0, K);

  struct Set {
    UnitRaw<FMT> g, u;
    u32x4 x[FM][4];
  };
  auto load = [&](Set& s, int step) {
    const int u = min(4 * step + g4, U - 1);
    s.g = load_unit<FMT, true>(wg, row, u, K);
    s.u = load_unit<FMT, true>(wu, row, u, K);
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
          p.h[at] = uint16_t(pack16<F16>(act_of(p.act, g[e]) * u[e], 0.f));
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
#ifndef VAR_CFG
#define VAR_CFG 4, 2, 2, 4
#define VAR_T 512
#endif
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, VAR_CFG>), dim3(unsigned(int64_t((p.N + 127) / 128) * ((p.M + 255) / 256))), dim3(VAR_T), 0,
                       s, p);
  } else {
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, 2, 2, 2, 2>), dim3(unsigned(int64_t((p.N + 63) / 64) * ((p.M + 127) / 128))), dim3(256), 0, s,
                       p);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace qmv
