// Backward pass of the gated products: dX = dG Wg + dU Wu, on the matrix cores.
#pragma once

#include <utility>

#include "gemm16.h"

namespace qmv {

struct GluBwdArgs {
  Mat wg, wu;
  const uint16_t *dg, *du;  // [M][ld], ld a multiple of 8; zeros where n >= N
  const uint16_t *dgl, *dul;  // WIDE: their low parts, laid out the same
  uint16_t* dx;
  float* part;              // [splits][M][K] partial sums, or null: one split, dx written
  int M, N, K, ld;
  int steps;                // stages per split, a multiple of 4
};

namespace {

// The decoded tile of a stage: 32 rows n of BR columns k, as the weights lie in
// memory.  The matrix cores want for each k eight consecutive n, which
// ds_read_b64_tr_b16 gathers: of 16 lanes, lanes 4 j .. 4 j + 3 name 16
// consecutive k of row j, and lane l receives the four rows' values of k = l.
// 64-byte blocks of a row (one unit) are exchanged by n % 4 and the 16-byte
// pieces of a pair by n / 4 % 2, which by the banks keeps apart both these reads
// (four rows of one unit) and the decoders' writes (rows n and n + 4 of 8 half
// units).  Conflicts are counted all the same, not traced to one of them: 0.74
// cycles per LDS instruction (8192 tokens, W4A16; 0.63 with low parts).
// In 16-byte pieces: row n, unit ul of the tile, half h, piece i.
template <int BR>
__device__ __forceinline__ int rows_at(int n, int ul, int h, int i) {
  return n * (BR / 8) + (ul ^ (n & 3)) * 4 + 2 * h + (i ^ ((n >> 2) & 1));
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ u32x2 read_tr(const u32x4* A, int pos8) {  // pos8: in 8-byte units
  lds_s16x4* p = (lds_s16x4*)(reinterpret_cast<const u32x2*>(A) + pos8);
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// Loads of load_half with a lane's unit, at least.
template <int FMT>
constexpr int kHalfLoads = FMT == QMV_Q6K ? 4 : is_fifth(FMT) ? 3 : 2;

// dX[m][k] = sum_n dG[m][n] W~g[n][k] + dU[m][n] W~u[n][k], one f32 accumulator
// over both sums.  The matrix cores take 16-bit operands.  Without WIDE these are
// dG and dU as they leave the call, rounded once: the relative error of dX is then
// about sqrt(2) of what rounding dX alone gives (more where the terms of a sum
// cancel), as in a model that trains in this type.  With WIDE a second token tile
// per stage holds what that rounding left over, rounded to the same type (dgates8),
// and is multiplied by the same weight fragments: twice the MFMAs, one decoding.
// W4A16, 5632 x 2048, the whole call: 24 tokens 20 us against 17, 512 tokens 74
// against 56, 8192 tokens 760 against 435 - 450 (there the large tile, at its
// register limit, spills some 20 values).
//
// RB, TB: 32-column blocks of dX and 32-token blocks per wave; WR x WT waves.
//
// The depth is n: first the gate rows, then the up rows, 32 to a stage.  Tokens
// (dG, dU) go straight from global memory into a ring of four LDS tiles, three
// stages ahead.  A thread decodes half a unit of one row per stage, from
// registers that were loaded six stages ahead, into the ring of weight tiles, two
// stages ahead (dense bf16 rows need no decoding and are copied like the
// tokens).  As in the forward kernel the first fragments of a stage are read
// before the barrier that ends the stage before it.
//
// Bound by the matrix cores and the decoding beside them: W4A16, 5632 x 2048,
// 8192 tokens take ~360 us, 1.05 PFLOP/s (a dense library product of the two
// matrices 290), MFMAs busy ~50 % of the SIMDs' cycles at 1.95 GHz.  The wider
// tile decodes a weight for 256 tokens; few tokens split the depth over
// workgroups instead (glu_backward_plan), as a stage's latency is then what counts.
template <int FMT, bool F16, bool WIDE, int RB, int TB, int WR, int WT>
__global__ __launch_bounds__(64 * WR * WT) void glu_bwd_kernel(const GluBwdArgs p) {
  constexpr int NT = 64 * WR * WT;
  constexpr int BR = 32 * RB * WR, BM = 32 * TB * WT;
  constexpr int XPT = BM * 4 / NT, APT = BR * 4 / NT;  // 16-byte pieces per thread and stage
  constexpr bool DIRECT = FMT == QMV_DENSE_BF16 && !F16;
  constexpr int P = WIDE ? 2 : 1;  // token tiles per stage: high parts, low parts
  static_assert(2 * BR == NT && XPT * NT == BM * 4 && APT * NT == BR * 4);

  __shared__ u32x4 A0[BR * 4], A1[BR * 4], A2[BR * 4], A3[BR * 4];
  __shared__ u32x4 X0[BM * 4], X1[BM * 4], X2[BM * 4], X3[BM * 4];
  asm volatile("" ::"v"(A0), "v"(A1), "v"(A2), "v"(A3) : "memory");  // escape, as in the forward kernel
  asm volatile("" ::"v"(X0), "v"(X1), "v"(X2), "v"(X3) : "memory");
  auto At = [&]<int S>() { return (S & 3) == 0 ? A0 : (S & 3) == 1 ? A1 : (S & 3) == 2 ? A2 : A3; };
  auto Xt = [&]<int S>() { return (S & 3) == 0 ? X0 : (S & 3) == 1 ? X1 : (S & 3) == 2 ? X2 : X3; };

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WT, wt = wave % WT;
  const TileId id0 = tile_of_block(p.K, BR, p.M, BM);
  const int k0 = id0.x * BR, m0 = id0.y * BM;
  const int N = p.N, K = p.K, U = K >> 5, ld = p.ld;
  const int NS = (N + 31) >> 5;  // stages per matrix
  const int first = blockIdx.y * p.steps, end = min(first + p.steps, 2 * NS);

  // this thread's half unit: of row nl of a stage, unit ul of the tile
  const int half = tid & 1;
  constexpr int UB = BR == 256 ? 1 : 0;  // bits of ul past the lowest two
  const int nr = tid >> (4 + UB);        // row bits 0, 1, 3, 4
  const int ul = ((tid >> 1) & 3) | (UB ? ((tid >> 4) & 1) * 4 : 0);
  const int nl = (nr & 3) | ((tid >> 3) & 1) * 4 | (nr >> 2) * 8;
  const int u = min((k0 >> 5) + ul, U - 1);
  // The weights of one stage after the other: first rows of the stage in every
  // plane, scalars that advance by 32 rows; the last stage again past the end.
  struct Walk {
    Mat m;
    int nb, t;
  };
  auto walk_from = [&](int t) {
    t = min(t, 2 * NS - 1);
    const bool up = t >= NS;
    Walk w;
    w.t = t;
    w.nb = 32 * (up ? t - NS : t);
#pragma unroll
    for (int i = 0; i < kPlanes<FMT>; ++i)
      w.m.p[i] = (up ? p.wu.p[i] : p.wg.p[i]) + int64_t(w.nb) * row_bytes<FMT>(i, K);
    return w;
  };
  auto advance = [&](Walk& w) {
    const bool stay = w.t + 1 >= 2 * NS, turn = w.t + 1 == NS;
    w.t += stay ? 0 : 1;
    w.nb = turn ? 0 : w.nb + (stay ? 0 : 32);
#pragma unroll
    for (int i = 0; i < kPlanes<FMT>; ++i)
      w.m.p[i] = turn ? p.wu.p[i] : w.m.p[i] + (stay ? 0 : 32 * row_bytes<FMT>(i, K));
  };
  const RowAt<FMT> nl_at = row_at<FMT>(nl, K);
  auto load = [&](const Walk& w) {
    RowAt<FMT> r;  // rows past N: the last one
    const uint32_t lastrow = N - 1 - w.nb;
#pragma unroll
    for (int i = 0; i < kPlanes<FMT>; ++i) r.o[i] = nl <= int(lastrow) ? nl_at.o[i] : lastrow * row_bytes<FMT>(i, K);
    return load_half<FMT, kByUnit>(w.m, r, u, half);
  };
  // Rows past N and stages past the end meet zero tokens, but an infinite weight
  // (f16: past 65504) times zero would be a NaN: their weights are zeros too.
  auto rows_of = [&](int t) { return t < end ? N - 32 * (t < NS ? t : t - NS) : 0; };
  auto decode = [&](const HalfRaw<FMT>& c, int i, u32x4* A) {
    A[rows_at<BR>(nl, ul, half, i)] = word_piece<FMT, F16>(c, u, 2 * half + i, i);
  };
  // dense rows: LDS slot tid + t * NT is row (tid + t * NT) / (BR / 8)
  uint32_t ao[APT];
  int an[APT];
#pragma unroll
  for (int t = 0; t < APT; ++t) {
    const int id = tid + t * NT, n = id / (BR / 8), s = id % (BR / 8);
    const int unit = min((k0 >> 5) + ((s >> 2) ^ (n & 3)), U - 1);
    ao[t] = 64 * unit + 32 * ((s >> 1) & 1) + 16 * ((s & 1) ^ ((n >> 2) & 1));
    an[t] = n;
  }
  auto copy_a = [&](const Walk& w, int stage, u32x4* A) {  // an offset past the buffer reads as zero
    const Buf b = buffer_of(scalar_base(w.m.p[0]), 0x7FFFFFFF);
    const int rows = rows_of(stage);
#pragma unroll
    for (int t = 0; t < APT; ++t)
      copy_to_lds(b, an[t] < rows ? uint32_t(an[t]) * uint32_t(2 * K) + ao[t] : 0x80000000u, 0, A + t * NT + wave * 64);
  };
  // Tokens: LDS slot tid + t * NT of a tile is row (tid + t * NT) / 4.  Pieces past
  // the row, and all pieces of a stage past the split's end, get an offset past
  // the buffer, which reads as zero.
  const uint8_t* gx = reinterpret_cast<const uint8_t*>(p.dg + int64_t(m0) * ld);
  const uint8_t* ux = reinterpret_cast<const uint8_t*>(p.du + int64_t(m0) * ld);
  const uint8_t* gw = WIDE ? reinterpret_cast<const uint8_t*>(p.dgl + int64_t(m0) * ld) : nullptr;
  const uint8_t* uw = WIDE ? reinterpret_cast<const uint8_t*>(p.dul + int64_t(m0) * ld) : nullptr;
  const int xc = (tid & 3) ^ ((tid >> 4) & 3);
  uint32_t xo[XPT];
#pragma unroll
  for (int t = 0; t < XPT; ++t)
    xo[t] = uint32_t(min(m0 + t * (NT / 4) + (tid >> 2), p.M - 1) - m0) * uint32_t(2 * ld) + 16 * xc;
  struct XWalk {
    const uint8_t *p, *l;
    int nb, t;
  };
  auto copy_x = [&]<int PART>(XWalk& w, u32x4* X) {  // and, behind a stage's last part, on to the next stage
    const bool in = w.t < end && w.nb + 8 * xc < ld;
    const Buf b = buffer_of(scalar_base(PART ? w.l : w.p), 0x7FFFFFFF);
#pragma unroll
    for (int t = 0; t < XPT; ++t) copy_to_lds(b, in ? xo[t] : 0x80000000u, 0, X + t * NT + wave * 64);
    if constexpr (PART == P - 1) {
      w.t += 1;
      const bool turn = w.t == NS;
      w.nb = turn ? 0 : w.nb + 32;
      w.p = turn ? ux : w.p + 64;
      if constexpr (WIDE) w.l = turn ? uw : w.l + 64;
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
  const int bj = (lane >> 2) & 3, bh = (lane >> 4) & 1, bc = lane & 3;  // transposing reads
  struct Frag {
    u32x4 a[RB], b[TB];
  };
  auto read_a = [&](Frag& f, const u32x4* A, int s) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int n = 16 * s + 8 * fh + bj;
      const u32x2 lo = read_tr(A, 2 * rows_at<BR>(n, wr * RB + i, bh, bc >> 1) + (bc & 1));
      const u32x2 hi = read_tr(A, 2 * rows_at<BR>(n + 4, wr * RB + i, bh, bc >> 1) + (bc & 1));
      f.a[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  };
  auto read_b = [&](Frag& f, const u32x4* X, int s) {
#pragma unroll
    for (int i = 0; i < TB; ++i) f.b[i] = X[tile32_at((wt * TB + i) * 32 + fr, 2 * s + fh)];
  };
  auto mul = [&](const Frag& f) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j) acc[i][j] = mfma32<F16>(f.a[i], f.b[j], acc[i][j]);
  };
  auto fence = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  HalfRaw<FMT> c[4];
  Walk walk = walk_from(first);
  const int64_t x0 = 64 * int64_t(first < NS ? first : first - NS);
  XWalk xwalk{(first < NS ? gx : ux) + x0, WIDE ? (first < NS ? gw : uw) + x0 : nullptr, int(x0 >> 1), first};
  auto copy_a_next = [&](int stage, u32x4* A) {
    copy_a(walk, stage, A);
    advance(walk);
  };
  auto load_next = [&] {
    const HalfRaw<FMT> r = load(walk);
    advance(walk);
    return r;
  };
  if constexpr (DIRECT) {
    copy_a_next(first, A0);
    copy_a_next(first + 1, A1);
    copy_a_next(first + 2, A2);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = load_next();
  }
  copy_x.template operator()<0>(xwalk, X0);
  copy_x.template operator()<1 % P>(xwalk, X1);
  copy_x.template operator()<2 % P>(xwalk, X2);
  if constexpr (!DIRECT) {
    keep_weights(c[0], nl < rows_of(first));
    keep_weights(c[1], nl < rows_of(first + 1));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      decode(c[0], i, A0);
      decode(c[1], i, A1);
    }
    c[0] = load_next();
    c[1] = load_next();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier16();
  Frag f0, f1;
  read_a(f0, A0, 0);
  read_b(f0, X0, 0);
#pragma unroll 1
  for (int st = first; st < end; st += 4) {
    [&]<int... H>(std::integer_sequence<int, H...>) {
      (([&] {
         // token tile H: part `part` of stage S; a stage's weight fragments serve both parts
         constexpr int S = H / P, part = H % P;
         u32x4* A2n = At.template operator()<S + 2>();
         copy_x.template operator()<(H + 3) % P>(xwalk, Xt.template operator()<H + 3>());
         if constexpr (DIRECT && part == 0) {
           if constexpr (WIDE) fence();  // the wait below counts on this order
           copy_a_next(st + S + 3, At.template operator()<S + 3>());
         }
         fence();
         if constexpr (part == 0) read_a(f1, At.template operator()<S>(), 1);
         read_b(f1, Xt.template operator()<H>(), 1);
         if constexpr (!DIRECT && part == 0) {
           keep_weights(c[(S + 2) & 3], nl < rows_of(st + S + 2));
           decode(c[(S + 2) & 3], 0, A2n);
         }
         mul(f0);
         fence();
         if constexpr (part == P - 1) read_a(f0, At.template operator()<S + 1>(), 0);
         read_b(f0, Xt.template operator()<H + 1>(), 0);
         if constexpr (!DIRECT && part == P - 1) {
           decode(c[(S + 2) & 3], 1, A2n);
           c[(S + 2) & 3] = load_next();
         }
         mul(f1);
         fence();
         // The next tile reads token tile H + 2 and, where it ends a stage, the weights of
         // the stage after its own.  Those tokens were copied in the tile before this one,
         // the weights in it or earlier.  Certainly issued after them: this tile's copies of
         // tokens and, of these two tiles, one (WIDE) or two stages' loads of codes; with
         // copied weights those of one stage, in this tile or behind the tokens of the last.
         asm volatile("s_waitcnt vmcnt(%0)" ::"n"(DIRECT ? XPT + APT : XPT + (WIDE ? 1 : 2) * kHalfLoads<FMT>)
                      : "memory");
         lds_barrier16();
       }()),
       ...);
    }(std::make_integer_sequence<int, 4 * P>{});
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the copies past the end
  lds_barrier16();

  // C fragment: lane holds columns k = 8 q + 4 fh + e (q, e in 0..3) of token lane % 32
  if (p.part) {
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
          *reinterpret_cast<f32x4*>(p.part + (int64_t(blockIdx.y) * p.M + m) * K + k) = v;
        }
    }
    return;
  }
  // through the wave's own part of LDS, 32 tokens x 64 columns at a time: rows leave whole
  static_assert(WR * WT * 32 * 8 <= 2 * BR * 4);
  u32x4* mine = (wave & 1 ? A1 : A0) + (wave >> 1) * (32 * 8);
#pragma unroll
  for (int j = 0; j < TB; ++j)
#pragma unroll
    for (int g = 0; g < RB; g += 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& v = acc[g + i][j];
          reinterpret_cast<u32x2*>(mine + tile_at(fr, 4 * i + q))[fh] =
              u32x2{pack16<F16>(v[4 * q], v[4 * q + 1]), pack16<F16>(v[4 * q + 2], v[4 * q + 3])};
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // written and read by this wave only
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 8) {
        const int r = r0 + (lane >> 3), pc = lane & 7;
        const int m = m0 + (wt * TB + j) * 32 + r, k = k0 + (wr * RB + g) * 32 + 8 * pc;
        if (m < p.M && k < K) *reinterpret_cast<u32x4*>(p.dx + int64_t(m) * K + k) = mine[tile_at(r, pc)];
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

template <int FMT, bool F16, bool WIDE>
hipError_t glu_bwd_start(const GluBwdArgs& p, const GluBwdPlan& plan, hipStream_t s) {
  const dim3 grid(unsigned(plan.tiles), unsigned(plan.splits));
  if (plan.tile == 2)
    hipLaunchKernelGGL((glu_bwd_kernel<FMT, F16, WIDE, 4, 2, 2, 4>), grid, dim3(512), 0, s, p);
  else if (plan.tile == 1)
    hipLaunchKernelGGL((glu_bwd_kernel<FMT, F16, WIDE, 2, 2, 2, 2>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((glu_bwd_kernel<FMT, F16, WIDE, 2, 1, 2, 2>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int FMT, bool F16>
hipError_t glu_bwd_go(const GluBwdArgs& p, const GluBwdPlan& plan, hipStream_t s) {
  return plan.low_bytes ? glu_bwd_start<FMT, F16, true>(p, plan, s) : glu_bwd_start<FMT, F16, false>(p, plan, s);
}

}  // namespace
}  // namespace qmv
