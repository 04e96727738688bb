// The gated products of many tokens, H = act(X Wg^T) * (X Wu^T), on the matrix cores.
#pragma once

#include <utility>

#include "gemm16.h"

namespace qmv {

struct GluFwdArgs {
  Mat wg, wu;
  const uint16_t* x;
  uint16_t *h, *g, *u;  // g, u may be null (both)
  int M, N, K, act;
};

namespace {

// How many vector memory operations a wave has certainly issued by the end of
// stage `now` after the copy of the tokens (or of the codes) in stage `from`.  A
// stage issues the XPT copies of its tokens, then, where it starts to decode a
// tile of codes, the CPT copies of the tile after the next, then, once per run,
// the loads of the next run's scales.
template <int FMT, int XPT, int CPT>
constexpr int issued_after(int from, bool codes, int now) {
  int n = 0;
  for (int s = from; s <= now; ++s) {
    const int h = (s + 4 * kRun) % kRun;
    if (s > from) n += XPT;
    if (s == from && codes) continue;  // the order of the scales' loads and the codes' copies is open
    if ((h + 2) % kChunk<FMT> == 0) n += CPT;
    if (h == 0) n += kMetaLoads<FMT>;
  }
  return n;
}

// Many tokens.  g = sum_k W~g[n][k] x[m][k] and u likewise in f32 accumulators,
// H = act(g) u rounded once; gate and up row n meet in one wave, so the product
// needs no second pass over G and U (which leave only if the caller keeps them
// for the backward pass).
//
// RB, TB: 32-row blocks of weights (half gate, half up) and of tokens per wave;
// KG groups of WR x WT waves.  Two groups halve K between them, each with tiles of
// its own, and the second's sums join the first's in LDS: where a unit has one
// small workgroup anyway, a second wave per SIMD works while the first waits.
//
// K goes by in stages of 32: one unit of every weight row and 64 bytes of every
// token, in a ring of four LDS tiles each.  Tokens go straight from global
// memory to LDS, three stages ahead (seven were no faster).  So do the weights'
// codes, 64 bytes of every row at a time into two more tiles; from there
// neighbouring threads decode one unit of a row into the operand type, once per
// workgroup, two stages ahead.  The first fragments of a stage are read before
// the barrier that ends the stage before it, so no wave waits for LDS behind a
// barrier (with 64-deep steps in two buffers, all read after the barrier, a step
// took 1.85 us for 0.92 us of MFMA).  Dense weights fill a tile of codes per stage:
// they are copied in the stage before the one that reads them, every stage ends
// with a wait for all copies, and nothing stays in flight over a barrier (512 tokens
// 41 us against W4A16's 35, 8192 tokens 408 against 366).
//
// Bound by the matrix cores and what shares their issue slots.  W4A16, 5632 x
// 2048: 8192 tokens with G and U kept take 365 - 394 us, 0.96 - 1.04 PFLOP/s (414
// where call follows call for long and the clock falls; a dense bf16 library
// product of the two matrices alone takes 393).  The MFMAs are busy 52 % of the
// SIMDs' cycles at the 1.86 GHz that the card holds under this load, LDS 30 %; the
// rest is the decoding (~24 VALU instructions per 8 weights), the barriers,
// ~26 us of stores, and units without work: 1408 tiles are 5.5 rounds of 256 units
// (busy 0.85 - 0.87 of the time).  512 tokens take 31 - 36 us, 0.65 - 0.77 PFLOP/s:
// 176 tiles, 0.69 of one round (units busy 0.50 of the time), and ~10 us of launch,
// first loads and epilogue.
template <int FMT, bool F16, int RB, int TB, int WR, int WT, int KG>
__global__ __launch_bounds__(64 * WR * WT * KG) void glu_fwd_kernel(const GluFwdArgs p) {
  constexpr int NT = 64 * WR * WT;      // threads of a group
  constexpr int BR = 32 * RB * WR, BN = BR / 2, BM = 32 * TB * WT;
  constexpr int XPT = BM * 4 / NT;      // 16-byte token pieces per thread and stage
  constexpr int SR = kRun, SC = kChunk<FMT>;  // stages per run and per tile of codes
  constexpr int CPT = BR * 4 / NT;      // ... of codes, per thread and tile
  constexpr int WPT = CPT;              // words of 8 weights that a thread decodes per stage
  static_assert((WPT == 1 || WPT == 2) && CPT * NT == BR * 4 && XPT * NT == BM * 4 && RB % 2 == 0);
  constexpr int XD = 3;                 // stages that the tokens' copies run ahead

  // variables of their own: the compiler then knows that a copy into one does
  // not concern the reads of the others
  __shared__ u32x4 SA0[KG][BR * 4], SA1[KG][BR * 4], SA2[KG][BR * 4], SA3[KG][BR * 4];
  __shared__ u32x4 SX0[KG][BM * 4], SX1[KG][BM * 4], SX2[KG][BM * 4], SX3[KG][BM * 4];
  __shared__ u32x4 SR0[KG][BR * 4], SR1[KG][BR * 4];  // rows of codes: gate 0 .. BN - 1, then up
  // let their addresses escape: otherwise the compiler knows that no asm
  // statement can touch them and moves LDS reads across the fences below
  asm volatile("" ::"v"(SA0), "v"(SA1), "v"(SA2), "v"(SA3) : "memory");
  asm volatile("" ::"v"(SX0), "v"(SX1), "v"(SX2), "v"(SX3), "v"(SR0), "v"(SR1) : "memory");
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  u32x4 *const A0 = SA0[kg], *const A1 = SA1[kg], *const A2 = SA2[kg], *const A3 = SA3[kg];
  u32x4 *const X0 = SX0[kg], *const X1 = SX1[kg], *const X2 = SX2[kg], *const X3 = SX3[kg];
  u32x4 *const R0 = SR0[kg], *const R1 = SR1[kg];
  auto At = [&]<int S>() { return (S & 3) == 0 ? A0 : (S & 3) == 1 ? A1 : (S & 3) == 2 ? A2 : A3; };
  auto Xt = [&]<int S>() { return (S & 3) == 0 ? X0 : (S & 3) == 1 ? X1 : (S & 3) == 2 ? X2 : X3; };

  const int tid = threadIdx.x - kg * NT, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WT, wt = wave % WT;
  const TileId id0 = tile_of_block(p.N, BN, p.M, BM);
  const int n0 = id0.x * BN, m0 = id0.y * BM;
  const int K = p.K, U = K >> 5;

  // 4 / WPT neighbouring threads decode a unit of a weight row, each the words
  // word .. word + WPT - 1: gate or up goes by wave, so that the addresses are
  // scalar bases and one lane offset per plane.
  const int word = tid % (4 / WPT) * WPT, half = word >> 1, ri = tid / (4 / WPT);
  const bool up = wave >= WR * WT / 2;
  const uint32_t wrow = min(n0 + ri % BN, p.N - 1) - n0;
  const Mat wg = from_row<FMT>(p.wg, n0, K), wu = from_row<FMT>(p.wu, n0, K), w = up ? wu : wg;
  // Codes: thread tid copies piece tid % 4 (by the tile's order) of gate and of up
  // row tid / 4, or of one of them where the threads cover both.
  const uint32_t co = uint32_t(min(n0 + (tid >> 2) % BN, p.N - 1) - n0) * row_bytes<FMT>(0, K) + 16 * ((tid & 3) ^ ((tid >> 4) & 3));
  const int arow = ((ri % BN) / (16 * RB)) * 32 * RB + (ri % BN) % (16 * RB) + (up ? 16 * RB : 0);
  // Token pieces: LDS slot tid + t * NT of a tile is row (tid + t * NT) / 4.
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x + int64_t(m0) * K);
  const Buf xbuf = buffer_of(xb), gbuf = buffer_of(wg.p[0]), ubuf = buffer_of(wu.p[0]);
  const Buf cbuf = buffer_of(scalar_base(w.p[0]));
  uint32_t xo[XPT];
#pragma unroll
  for (int t = 0; t < XPT; ++t)
    xo[t] = uint32_t(min(m0 + t * (NT / 4) + (tid >> 2), p.M - 1) - m0) * uint32_t(2 * K) +
            16 * ((tid & 3) ^ ((tid >> 4) & 3));

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
  auto read = [&](Frag& f, const u32x4* A, const u32x4* X, int s) {
#pragma unroll
    for (int i = 0; i < RB; ++i) f.a[i] = A[tile32_at((wr * RB + i) * 32 + fr, 2 * s + fh)];
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
  auto copy_x = [&](int u, u32x4* X) {  // unit u of the tokens
#pragma unroll
    for (int t = 0; t < XPT; ++t) copy_to_lds(xbuf, xo[t], 64 * u, X + t * NT + wave * 64);
  };

  auto copy_codes = [&](int u, u32x4* R) {  // units u .. u + SC - 1
    if constexpr (CPT == 2) {
      copy_to_lds(gbuf, co, u * (64 / SC), R + wave * 64);
      copy_to_lds(ubuf, co, u * (64 / SC), R + BN * 4 + wave * 64);
    } else {
      copy_to_lds(cbuf, co, u * (64 / SC), R + wave * 64);
    }
  };

  // ---- whole runs
  const int all = U / SR, per = (all + KG - 1) / KG;
  const int r0 = kg * per, runs = min(per, all - r0);  // this group's, from r0 on
  const int idle = per - runs;
  if (runs > 0) {
    // Workgroups start at different runs: in step they would all read the same
    // columns of rows a power of two apart, which lie on few L2 channels.
    int ua = (r0 + id0.y % runs) * SR;  // first unit of the current run
    RunMeta<FMT> cur, next;
    // words i of the unit of stage s of a run (first unit u, scales x) from codes R
    auto decode = [&](const u32x4 (&codes)[2], const RunMeta<FMT>& x, int u, int s, u32x4* A, int i) {
      HalfRaw<FMT> r;
      r.q[0] = codes[0];
      r.q[1] = codes[1];
      meta_of<FMT>(r, x, s);
      A[tile32_at(arow, word + i)] = word_piece<FMT, F16>(r, u + s, word + i, i);
    };
    // Tile of codes of stage s (of this run or, past SR, the next).
    auto Rt = [&]<int S>() { return (S / SC) & 1 ? R1 : R0; };
    cur = load_run_meta<FMT>(w, wrow, ua, half, K);
    copy_codes(ua, R0);
    copy_codes(ua + SC, R1);
    [&]<int... S>(std::integer_sequence<int, S...>) {
      (copy_x(ua + S, Xt.template operator()<S>()), ...);
    }(std::make_integer_sequence<int, XD>{});
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier16();
    [&]<int... S>(std::integer_sequence<int, S...>) {
      (([&] {
         u32x4 c[2];
         read_codes<FMT, WPT>(c, Rt.template operator()<S>(), ri, S % SC, word);
#pragma unroll
         for (int i = 0; i < WPT; ++i) decode(c, cur, ua, S, S ? A1 : A0, i);
       }()),
       ...);
    }(std::make_integer_sequence<int, 2>{});
    lds_barrier16();
    if constexpr (SC == 1) {  // both tiles of codes are used up
      copy_codes(ua + 2, R0);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      lds_barrier16();
    }
    Frag f0, f1;
    u32x4 c[2][2];
    read(f0, A0, X0, 0);
    if constexpr (SC == 4) read_codes<FMT, WPT>(c[0], R0, ri, 2, word);
#pragma unroll 1
    for (int run = 0; run < runs; ++run) {
      const int then = ua + SR < (r0 + runs) * SR ? ua + SR : r0 * SR;
      [&]<int... H>(std::integer_sequence<int, H...>) {
        (([&] {
           const u32x4 *A = At.template operator()<H>(), *X = Xt.template operator()<H>();
           const u32x4 *A1n = At.template operator()<H + 1>(), *X1n = Xt.template operator()<H + 1>();
           u32x4* A2n = At.template operator()<H + 2>();
           // The stage decoded here is H + 2.  When it is the first of its tile of
           // codes, the other tile is done with: its next codes (those behind this
           // tile's) go there.
           constexpr int D = H + 2;
           constexpr bool fresh = D % SC == 0;
           constexpr int NC = D + SC;  // first stage of the codes to copy
           copy_x(H + XD < SR ? ua + H + XD : then + H + XD - SR, Xt.template operator()<H + XD>());
           fence();
           if constexpr (fresh) copy_codes(NC < SR ? ua + NC : NC < 2 * SR ? then + NC - SR : 0, Rt.template operator()<NC>());
           fence();
           if constexpr (H == 0) next = load_run_meta<FMT>(w, wrow, then, half, K);
           // Where a tile of codes lasts four stages, a stage's codes are read in the
           // stage before.
           if constexpr (SC < 4) read_codes<FMT, WPT>(c[H & 1], Rt.template operator()<D>(), ri, D % SC, word);
           read(f1, A, X, 1);
           auto dec = [&](int i) {
             if constexpr (D >= SR) decode(c[H & 1], next, then, D - SR, A2n, i);
             else decode(c[H & 1], cur, ua, D, A2n, i);
           };
           dec(0);
           mul(f0);
           fence();
           read(f0, A1n, X1n, 0);
           if constexpr (SC == 4) read_codes<FMT, WPT>(c[(H + 1) & 1], Rt.template operator()<D + 1>(), ri, (D + 1) % SC, word);
           if constexpr (WPT == 2) dec(1);
           mul(f1);
           fence();
           // The next stage reads the tokens of stage H + 2, and the codes of the stage
           // `code`, if they start a tile.  Everything issued after their copies may
           // still be under way.
           constexpr int code = SC == 4 ? H + 4 : H + 3;
           constexpr int left_x = issued_after<FMT, XPT, CPT>(H + 2 - XD, false, H);
           constexpr int left_c = code % SC ? 63 : issued_after<FMT, XPT, CPT>(code - SC - 2, true, H);
           constexpr int left = left_x < left_c ? left_x : left_c;
           static_assert(left >= 0 && left <= 63);
           asm volatile("s_waitcnt vmcnt(%0)" ::"n"(left) : "memory");
           lds_barrier16();
         }()),
         ...);
      }(std::make_integer_sequence<int, SR>{});
      cur = next;
      ua = then;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the copies past the end
    lds_barrier16();
  } else if (per > 0) {  // a single run is the first group's: the barriers outside its stages
    lds_barrier16();
    lds_barrier16();
    if constexpr (SC == 1) lds_barrier16();
    lds_barrier16();
  }
  // the barriers of the stages that the other group has more
  if constexpr (KG > 1)
    for (int i = 0; i < idle * SR; ++i) lds_barrier16();

  // ---- the rest of K, one unit at a time
  for (int u0 = all * SR; u0 < U; u0 += KG) {
    const int u = min(u0 + kg, U - 1);
#pragma unroll
    for (int t = 0; t < XPT; ++t) X0[tid + t * NT] = load_at<u32x4>(xb, xo[t] + 64 * u);
    const HalfRaw<FMT> r = load_half<FMT, kByRow>(w, row_at<FMT>(wrow, K), u, half);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (WPT == 2 || i == (word & 1)) A0[tile32_at(arow, 2 * half + i)] = word_piece<FMT, F16>(r, u, 2 * half + i, i);
    lds_barrier16();
    if (u0 + kg < U) {
      Frag f;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        read(f, A0, X0, s);
        mul(f);
      }
    }
    lds_barrier16();
  }

  // C fragment: lane holds rows n = 8 q + 4 fh + e (q, e in 0..3) of token
  // lane % 32.  Each output goes through the wave's own part of LDS (the tiles
  // are done with), so that rows of up to 128 bytes leave whole.
  lds_barrier16();
  if constexpr (KG == 2) {  // the second group's sums join the first's, through the second's tiles
    static_assert(RB * TB == 2 && NT * 2 == BR * 4);
    f32x4* const at[4] = {reinterpret_cast<f32x4*>(SA0[1]), reinterpret_cast<f32x4*>(SA1[1]),
                          reinterpret_cast<f32x4*>(SA2[1]), reinterpret_cast<f32x4*>(SA3[1])};
    if (kg == 1) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const f32x16& v = acc[c >> 2][0];
        at[c >> 1][(c & 1) * NT + tid] = f32x4{v[4 * (c & 3)], v[4 * (c & 3) + 1], v[4 * (c & 3) + 2], v[4 * (c & 3) + 3]};
      }
    }
    lds_barrier16();
    if (kg == 1) return;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const f32x4 v = at[c >> 1][(c & 1) * NT + tid];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[c >> 2][0][4 * (c & 3) + e] += v[e];
    }
  }
  constexpr int HB = RB / 2;                       // 32-row blocks of outputs
  constexpr int WPA = BR * 4 / (32 * 8);           // waves per weight tile, 32 tokens x 64 values each
  static_assert(NT / 64 <= 4 * WPA);
  const int wa = wave / WPA;
  u32x4* mine = (wa == 0 ? A0 : wa == 1 ? A1 : wa == 2 ? A2 : A3) + wave % WPA * (32 * 8);
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

// Few tokens: a weight stream.  A workgroup owns 16 FN gate and the same up
// rows; its W waves split K in steps of 128 (wave w takes steps w, w + W, ...,
// two of them in flight).  Lane group g (16 lanes) of a fragment holds one 32-k
// unit, word s of it being k = 32 g + 8 s .. + 7 of MFMA s; the token operand
// follows the same order straight from global memory (no two waves share a
// step, so LDS would only be a detour).  The partial tiles meet in LDS and are
// added in wave order.
//
// Bound by the latency of a chain that is only K / (128 W) steps long: Q4K,
// 5632 x 2048, 16 tokens take 9.7 us for 13.2 MB (1.37 TB/s; a copy of that size
// at the card's 5.1 TB/s would take 2.6), of which ~3 us is the launch.
template <int FMT, bool F16, int FM, int FN, int W>
__global__ __launch_bounds__(64 * W) void glu_fwd_few_kernel(const GluFwdArgs p) {
  constexpr int T = 2 * FN * FM;  // partial 16 x 16 tiles per wave
  __shared__ f32x4 red[W][T][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g4 = lane >> 4;
  const int n0 = blockIdx.x * 16 * FN, m0 = blockIdx.y * 16 * FM;
  const int K = p.K, U = K >> 5, nk = (K + 127) >> 7;
  const Mat wg = from_row<FMT>(p.wg, n0, K), wu = from_row<FMT>(p.wu, n0, K);
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x + int64_t(m0) * K);

  struct Set {
    UnitRaw<FMT> w[2][FN];
    u32x4 x[FM][4];
  };
  auto load = [&](Set& s, int step) {
    const int u = min(4 * step + g4, U - 1);
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const uint32_t row = min(n0 + 16 * i + fr, p.N - 1) - n0;
      s.w[0][i] = load_unit<FMT, kByUnit>(wg, row, u, K);
      s.w[1][i] = load_unit<FMT, kByUnit>(wu, row, u, K);
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const uint32_t m = min(m0 + 16 * j + fr, p.M - 1) - m0;
#pragma unroll
      for (int i = 0; i < 4; ++i) s.x[j][i] = load_at<u32x4>(xb, m * uint32_t(2 * K) + 64 * u + 16 * i);
    }
  };
  f32x4 acc[2][FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[0][i][j] = acc[1][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto use_as = [&]<bool WHOLE>(const Set& s, int step) {
    const int u = 4 * step + g4;
    const bool in = WHOLE || u < U;
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 b[FM];
#pragma unroll
      for (int j = 0; j < FM; ++j) b[j] = in ? s.x[j][i] : zero;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int n = 0; n < FN; ++n) {
          const u32x4 v = unit_piece<FMT, F16>(s.w[t][n], affine_of<FMT>(s.w[t][n].m, WHOLE ? u : min(u, U - 1)), i);
          const u32x4 a = in ? v : zero;
#pragma unroll
          for (int j = 0; j < FM; ++j) acc[t][n][j] = mfma16<F16>(a, b[j], acc[t][n][j]);
        }
    }
  };
  // only the last step can end inside
  auto use = [&](const Set& s, int step) {
    if (4 * step + 4 <= U) use_as.template operator()<true>(s, step);
    else use_as.template operator()<false>(s, step);
  };
  Set s0, s1;
  load(s0, wave);
  if (wave + W < nk) load(s1, wave + W);
  for (int st = wave; st < nk; st += 2 * W) {
    use(s0, st);
    if (st + 2 * W < nk) load(s0, st + 2 * W);
    if (st + W < nk) use(s1, st + W);
    if (st + 3 * W < nk) load(s1, st + 3 * W);
  }
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) red[wave][(i * FM + j) * 2 + t][lane] = acc[t][i][j];
  lds_barrier16();
  // C fragment: lane holds rows n0 + 16 i + 4 g4 + e of token fr
  for (int ij = wave; ij < FN * FM; ij += W) {
    f32x4 g = red[0][2 * ij][lane], u = red[0][2 * ij + 1][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      g += red[w][2 * ij][lane];
      u += red[w][2 * ij + 1][lane];
    }
    const int m = m0 + 16 * (ij % FM) + fr;
    if (m < p.M) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int nn = n0 + 16 * (ij / FM) + 4 * g4 + e;
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

// The fewest tokens: as above with 8 gate and the same 8 up rows in one fragment,
// which halves what a wave has to decode one after the other and gives twice the
// workgroups; every workgroup reads all tokens, so it pays for few of them only.
// W4A16, 5632 x 2048, one token: 7.4 us for 13 MB (1.76 TB/s).
template <int FMT, bool F16, int W>
__global__ __launch_bounds__(64 * W) void glu_fwd_fewest_kernel(const GluFwdArgs p) {
  __shared__ f32x4 red[W][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g4 = lane >> 4;
  const int n0 = blockIdx.x * 8;
  const int K = p.K, U = K >> 5, nk = (K + 127) >> 7;
  const uint32_t row = min(n0 + (fr & 7), p.N - 1) - n0;
  Mat w = from_row<FMT>(p.wg, n0, K);
  const Mat wu = from_row<FMT>(p.wu, n0, K);
#pragma unroll
  for (int i = 0; i < kPlanes<FMT>; ++i) w.p[i] = fr < 8 ? w.p[i] : wu.p[i];
  const uint32_t xrow = uint32_t(min(fr, p.M - 1)) * uint32_t(2 * K);
  const uint8_t* xb = reinterpret_cast<const uint8_t*>(p.x);
  struct Set {
    UnitRaw<FMT> w;
    u32x4 x[4];
  };
  auto load = [&](Set& s, int step) {
    const int u = min(4 * step + g4, U - 1);
    s.w = load_unit<FMT, kByMatrix>(w, row, u, K);
#pragma unroll
    for (int i = 0; i < 4; ++i) s.x[i] = load_at<u32x4>(xb, xrow + 64 * u + 16 * i);
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto use_as = [&]<bool WHOLE>(const Set& s, int step) {
    const int u = 4 * step + g4;
    const bool in = WHOLE || u < U;
    const u32x4 zero = {0, 0, 0, 0};
    const Affine f = affine_of<FMT>(s.w.m, WHOLE ? u : min(u, U - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 v = unit_piece<FMT, F16>(s.w, f, i);
      acc = mfma16<F16>(in ? v : zero, in ? s.x[i] : zero, acc);
    }
  };
  // only the last step can end inside
  auto use = [&](const Set& s, int step) {
    if (4 * step + 4 <= U) use_as.template operator()<true>(s, step);
    else use_as.template operator()<false>(s, step);
  };
  Set s0, s1;
  load(s0, wave);
  if (wave + W < nk) load(s1, wave + W);
  for (int st = wave; st < nk; st += 2 * W) {
    use(s0, st);
    if (st + 2 * W < nk) load(s0, st + 2 * W);
    if (st + W < nk) use(s1, st + W);
    if (st + 3 * W < nk) load(s1, st + 3 * W);
  }
  red[wave][lane] = acc;
  lds_barrier16();
  if (wave) return;
  f32x4 v = red[0][lane];
#pragma unroll
  for (int w = 1; w < W; ++w) v += red[w][lane];
  // lanes 0 .. 31 hold gate rows n0 + 4 g4 + e of token fr, lanes 32 .. 63 the same up rows
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float u = __shfl_xor(v[e], 32);
    const int n = n0 + 4 * g4 + e;
    if (lane < 32 && fr < p.M && n < p.N) {
      const int64_t at = int64_t(fr) * p.N + n;
      p.h[at] = uint16_t(pack16<F16>(act_of(p.act, v[e]) * u, 0.f));
      if (p.g) {
        p.g[at] = uint16_t(pack16<F16>(v[e], 0.f));
        p.u[at] = uint16_t(pack16<F16>(u, 0.f));
      }
    }
  }
}

template <int FMT, bool F16>
hipError_t glu_fwd_go(const GluFwdArgs& p, hipStream_t s) {
  // More rows per workgroup read the tokens fewer times, fewer rows keep more
  // workgroups at work: 16 + 16 rows as long as these are one round of the chip (256
  // units), 32 + 32 past it.  W4A16, K = 2048, us with 8 + 8 / 16 + 16 / 32 + 32 rows:
  //   N            2048             4096             5632             8192
  //    1 token   4.4  5.6  8.1    5.7  5.7  8.2    7.5  7.8  8.3    8.8  7.9  8.3
  //   16 tokens  5.6  6.7  9.3    8.4  6.9  9.4   11.0 10.3  9.4   13.6 10.5  9.5
  //   32 tokens       8.6 11.2         8.7 11.3        15.2 11.4        15.2 11.5
  //   64 tokens      12.6 17.6        12.8 17.6        24.1 17.9        24.2 18.2
  // Q6K at N = 4096, 16 and 64 tokens, 8.3 and 14.2 with 16 + 16 against 12.0 and 20.2.
  // Over 320 sizes of five formats (N 2048 to 14336, 1 to 64 tokens) the choice is 5 %
  // over the best on average; worst where 64 x 64 tiles would do better, 33 to 64
  // tokens of very wide matrices (14336 x 4096, 64 tokens: 56 against 33).
  if (p.M <= 16 && int64_t(p.M) * p.N <= 24576) {
    hipLaunchKernelGGL((glu_fwd_fewest_kernel<FMT, F16, 8>), dim3((p.N + 7) / 8), dim3(512), 0, s, p);
    return hipGetLastError();
  }
  const int64_t blocks = (p.M + 63) / 64, few = int64_t((p.N + 15) / 16) * blocks;
  if (p.M <= 64 || few <= 256) {
    const bool wide = p.M <= 64 && p.N > 4096;
    const dim3 grid(unsigned(wide ? (p.N + 31) / 32 : (p.N + 15) / 16), unsigned(blocks));
    if (p.M <= 16 && wide)
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 1, 2, 8>), grid, dim3(512), 0, s, p);
    else if (p.M <= 16)
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 1, 1, 8>), grid, dim3(512), 0, s, p);
    else if (p.M <= 32 && wide)
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 2, 2, 8>), grid, dim3(512), 0, s, p);
    else if (p.M <= 32)
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 2, 1, 8>), grid, dim3(512), 0, s, p);
    else if (wide)
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 4, 2, 4>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((glu_fwd_few_kernel<FMT, F16, 4, 1, 4>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
  }
  // A launch takes rounds of the chip: the smallest tile is taken whose count is
  // one round (256 units, two 64 x 128 tiles to a unit), else the largest, which
  // decodes a weight once for the most tokens.  Us on W4A16, K = 2048, for tiles of
  // outputs x tokens:        64 x 64   64 x 128   64 x 256   128 x 256
  //   N 5632,  128 tokens       20        24         31         47
  //            256 tokens       38        26         31         47
  //            512 tokens       59        41         34         50
  //           1024 tokens      113        73         68         56
  // Over 315 sizes of seven formats (N 1333 to 14336, 96 to 2048 tokens) 0.5 % over the
  // best tile on average, at most 12 % (Q6K, 14336 x 4096, 768 tokens: 238 against 212).
  // The few-token kernel up to 256 groups, the 64 x 64 tile past them: Q4K, 1024 x
  // 1024, 128 tokens (128 groups) 7.9 against 11.0; W4A16, 1333 x 768, 197 tokens
  // (336) 12.8 against 10.8; 5632 x 2048, 128 tokens (704) 38 against 20.
  // Two groups of waves from K = 1024 on (four runs): W4A16, 2048 wide, 256 tokens
  // 19.3 against 21.8 at K = 2048, 15.7 against 17.3 at 1536; 1333 wide, 197 tokens
  // 11.4 against 12.6 at 1024, 10.4 both at 768 (Q6K 14.1 against 13.3); 1300 wide,
  // 300 tokens 6.5 against 6.1 at 256.
  auto tiles = [&](int bn, int bm) { return int64_t((p.N + bn - 1) / bn) * ((p.M + bm - 1) / bm); };
  if (tiles(64, 64) <= 256 && p.K >= 1024)
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, 2, 1, 2, 2, 2>), dim3(unsigned(tiles(64, 64))), dim3(512), 0, s, p);
  else if (tiles(64, 64) <= 256)
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, 2, 1, 2, 2, 1>), dim3(unsigned(tiles(64, 64))), dim3(256), 0, s, p);
  else if (tiles(64, 128) <= 256 || (tiles(64, 256) > 256 && tiles(64, 128) <= 512))
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, 2, 1, 2, 4, 1>), dim3(unsigned(tiles(64, 128))), dim3(512), 0, s, p);
  else if (tiles(64, 256) <= 256)
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, 2, 2, 2, 4, 1>), dim3(unsigned(tiles(64, 256))), dim3(512), 0, s, p);
  else
    hipLaunchKernelGGL((glu_fwd_kernel<FMT, F16, 4, 2, 2, 4, 1>), dim3(unsigned(tiles(128, 256))), dim3(512), 0, s, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace qmv
