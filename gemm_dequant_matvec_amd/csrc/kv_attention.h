// Attention over the quantised cache: the kernel, as a template over the cache's
// format, the type and the head's size (kv_attention*.hip hold the instances).
//
//   s = scale K q,  p = 2^(s log2 e - ref),  o = V^T p / sum p
//
// transposed, so that a column of every matrix product is one query: S^T = K Q^T
// leaves a lane with 4 + 4 tokens of one query, which is what the operand P^T of
// O^T = V^T P^T wants of that lane (the order of the 32 tokens in the product is
// free, and V's lanes hold the same ones: the cache's layout).  So scores become
// probabilities and operands without leaving their lane, and the maximum and sum of
// a query need only the four lanes of its column.
//
// The codes are exact in f16 (1024 + code is a byte under 0x64, less 1152 or 1032),
// K's scale multiplies the f32 sums over a block of 32 dimensions and V's scale
// multiplies the probabilities, once for every block.  q is multiplied by a power of
// two so that its largest value lies in [2^14, 2^15): 16-bit queries are then exact in
// f16 and f32 ones, as two f16 parts, to 2^-22.
//
// p times V's scale has to be an f16 value (or two parts).  The exponent's reference
// takes care of the range: it is the running maximum plus the binary exponent of the
// largest V scale beside it, less 7, so that products start at 2^7 at most and are
// rescaled when one could pass 2^15; probabilities down to 2^-21 of the largest are
// normal f16 values then, and the reference cancels in o.  Raising it is a branch
// that few steps take.
//
// A workgroup of four waves takes 16 * TILES queries of one k / v head and a range of
// tokens, which its waves share in steps of 32 tokens; each wave keeps a running
// reference, sum and accumulator, and they meet in LDS at the end.  With few queries
// the tokens are split over workgroups too, whose results a second launch joins in a
// fixed order.
#pragma once

#include <algorithm>

#include "cache_internal.h"
#include "gemm16.h"

namespace qmv {

struct KvAttnArgs {
  KvArgs kv;
  const void* q;
  void* out;
  float* lse;
  float* sums;    // [T][q_heads][slots][D], workspace
  float2* stats;  // [T][q_heads][slots]: reference and sum
  int64_t q_token, q_head, out_token, out_head;
  float scale;    // times log2 e
  int group, q_heads, window, prefix, slots;
};

namespace {

constexpr float kInf = __builtin_inff();

template <int CTRL>
__device__ __forceinline__ int dpp_of(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
// f of the values of lane and lane ^ 16, then of lane ^ 32: over the four lanes of a column.
template <class T, class F>
__device__ __forceinline__ T over_column(T v, F f) {
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  const T two = f(__builtin_bit_cast(T, uint32_t(a[0])), __builtin_bit_cast(T, uint32_t(a[1])));
  const uint32_t y = __builtin_bit_cast(uint32_t, two);
  const auto b = __builtin_amdgcn_permlane32_swap(y, y, false, false);
  return f(__builtin_bit_cast(T, uint32_t(b[0])), __builtin_bit_cast(T, uint32_t(b[1])));
}
// Largest value of 16 lanes, in each of them.
__device__ __forceinline__ int row_max(int v) {
  v = max(v, dpp_of<0xB1>(v));
  v = max(v, dpp_of<0x4E>(v));
  v = max(v, dpp_of<0x141>(v));
  return max(v, dpp_of<0x140>(v));
}
// Of the wave, in every lane.
__device__ __forceinline__ int wave_max(int v) {
  return __builtin_amdgcn_readfirstlane(over_column(row_max(v), [](int a, int b) { return max(a, b); }));
}
__device__ __forceinline__ float column_max(float v) {
  return over_column(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float column_sum(float v) {
  return over_column(v, [](float a, float b) { return a + b; });
}

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Two code bytes of w as two f16 values code - BIAS: SEL names the bytes.
template <int BIAS>
__device__ __forceinline__ uint32_t codes16(uint32_t w, uint32_t sel) {
  const f16x2 v = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w, sel));
  const f16x2 b = {_Float16(1024 + BIAS), _Float16(1024 + BIAS)};
  return __builtin_bit_cast(uint32_t, v - b);
}

__device__ __forceinline__ float half_of(u32x2 w, int r) {
  const uint32_t bits = w[r >> 1];
  return f16_bits_to_f32(bits >> (16 * (r & 1)) & 0xFFFFu);
}

// A row of q: token r / group and head r % group of the k / v head, for row r of a sequence
// (or, for the shared prefix, of the whole call).
struct Row {
  int token;   // row of q, -1: none
  int head;    // of q
  int lo, hi;  // positions that it sees, lo .. hi - 1
};

// The sequence of each lane's token, for tokens of the whole call from `least` on (uniform) up: the
// wave finds that of the first, takes the starts of the 64 from there on, and each lane searches
// them; what lies further (past many sequences without rows) is found by bisection.
struct Sequences {
  int first, starts;  // starts: row start of sequence first + lane
  __device__ __forceinline__ void look_up(const KvArgs& kv, int least, int lane) {
    first = kv_search(kv.B, least, [&](int i) { return int64_t(kv_row_start(kv, i)); });
    starts = kv_row_start(kv, min(first + lane, kv.B));
  }
  __device__ __forceinline__ int of(const KvArgs& kv, int token) const {  // by a whole wave
    int x = 0;
#pragma unroll
    for (int h = 32; h > 0; h >>= 1)
      if (__shfl(starts, x + h) <= token && first + x + h < kv.B) x += h;
    int at = first + x;
    if (x == 63) {
      int n = kv.B - at;
      while (n > 1) {
        const int h = n >> 1;
        if (kv_row_start(kv, at + h) <= token) at += h, n -= h;
        else n = h;
      }
    }
    return at;
  }
};

// Called by a whole wave; seq: for the prefix.
template <bool PREFIX>
__device__ __forceinline__ Row row_of(const KvAttnArgs& a, const Sequences& seq, uint32_t r, uint32_t rows, int kv_head,
                                      int first_row, int64_t first_pos, int from, int64_t cap) {
  const int i = int(min(r, rows - 1) / uint32_t(a.group));
  Row w;
  w.token = first_row + i;
  w.head = kv_head * a.group + int(min(r, rows - 1)) - i * a.group;
  int64_t pos;
  bool there = r < rows;
  if constexpr (PREFIX) {
    const int x = seq.of(a.kv, w.token), start = kv_row_start(a.kv, x), end = kv_row_start(a.kv, x + 1);
    pos = int64_t(a.kv.kv_len[x]) - end + w.token;
    there = there && w.token >= start && w.token < end;
  } else {
    pos = first_pos + i;
  }
  const int64_t lo = a.window ? max(int64_t(0), pos - a.window + 1) : 0;
  w.lo = int(min(max(lo, int64_t(from)), cap));
  w.hi = int(max(int64_t(0), min(pos + 1, cap)));
  return there ? w : Row{-1, 0, 0, 0};
}

// The rows and positions that a workgroup works on: a sequence's own, or the prefix's.
struct Span {
  int kv_head, split, r0;
  uint32_t rows;
  int64_t first_pos, cap;
  const int32_t* table;
};
template <bool PREFIX>
__device__ __forceinline__ Span span_of(const KvAttnArgs& a, int splits) {
  const KvArgs& kv = a.kv;
  Span s;
  const int item = blockIdx.x / kv.heads, b = PREFIX ? 0 : item / splits;
  s.kv_head = blockIdx.x - item * kv.heads;
  s.split = item - b * splits;
  s.r0 = PREFIX ? 0 : kv_row_start(kv, b);
  const int r1 = PREFIX ? kv_row_start(kv, kv.B) : max(s.r0, kv_row_start(kv, b + 1));
  s.rows = uint32_t(r1 - s.r0) * uint32_t(a.group);  // below 2^31
  const int64_t cap = int64_t(kv.columns) * kv.sets * 16;
  s.cap = PREFIX ? min(cap, int64_t(a.prefix)) : cap;
  s.first_pos = PREFIX ? 0 : int64_t(kv.kv_len[b]) - (r1 - s.r0);
  s.table = kv.table + (PREFIX ? 0 : b * kv.stride);
  return s;
}

// What a split takes of the sets s0 .. s1 - 1: [u0, u1).  Shares are whole steps of `unit`
// sets, and `least` sets at least, so that short sequences end with fewer parts.  Many rows, 128 of each of 8
// heads of 128 over 600 tokens (Q8_0, bf16): parts of 256 tokens 22 us the call, of 128 18, of 64 17; over 4000: 28,
// 25.5 and 31.
constexpr int kLeastFew = 16, kLeastMany = 8;
__device__ __forceinline__ void share_of(int s0, int s1, int splits, int split, int unit, int least, int& u0, int& u1) {
  const int share = (max((s1 - s0 + splits - 1) / splits, least) + unit - 1) / unit * unit;
  u0 = int(min(int64_t(s1), s0 + int64_t(split) * share));
  u1 = min(s1, u0 + share);
}

// 16 * TILES queries of a wave: operands, running reference, sum and accumulator.
template <int E, int NB, int TILES>
struct Rows {
  static constexpr int QP = E == 0 ? 2 : 1;  // f16 parts of q
  static constexpr int PP = E == 2 ? 1 : 2;  // of a probability times scale

  u32x4 q[TILES][NB][QP];
  f32x4 o[TILES][NB][2];
  float factor[TILES], ref[TILES], sum[TILES];
  int lo[TILES], hi[TILES];
  int all_lo, all_hi;  // every row sees all_lo .. all_hi - 1
  int any_lo, any_hi;  // no row sees anything outside any_lo .. any_hi - 1

  // What the rows see, and nothing of it yet.
  __device__ __forceinline__ void begin(const Row (&row)[TILES]) {
    int most_lo = 0, least_hi = 0x7FFFFFFF, least_lo = 0x7FFFFFFF, most_hi = 0;
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const bool there = row[j].token >= 0;
      lo[j] = there ? row[j].lo : 0;
      hi[j] = there ? row[j].hi : 0x7FFFFFFF;
      most_lo = max(most_lo, lo[j]);
      least_hi = min(least_hi, hi[j]);
      if (there && lo[j] < hi[j]) {
        least_lo = min(least_lo, lo[j]);
        most_hi = max(most_hi, hi[j]);
      }
      ref[j] = -kInf;
      sum[j] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < 2; ++m) o[j][b][m] = f32x4{0, 0, 0, 0};
    }
    all_lo = wave_max(most_lo);
    all_hi = -wave_max(-least_hi);
    any_lo = -wave_max(-least_lo);
    any_hi = wave_max(most_hi);
    if (any_lo >= any_hi) any_lo = any_hi = 0;
  }

  // q is fetched before the tokens and made into operands while they are on their way.
  struct Fetched {
    u32x4 w[NB][E == 0 ? 2 : 1];
  };
  static __device__ __forceinline__ void fetch_q(const KvAttnArgs& a, const Row& row, int lane, Fetched& f) {
    const int64_t at = row.token * a.q_token + row.head * a.q_head + 8 * (lane >> 4);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int i = 0; i < (E == 0 ? 2 : 1); ++i) f.w[b][i] = u32x4{0, 0, 0, 0};
      if (row.token >= 0) {
        if constexpr (E == 0) __builtin_memcpy(f.w[b], static_cast<const float*>(a.q) + at + 32 * b, 32);
        else f.w[b][0] = load8(static_cast<const uint16_t*>(a.q) + at + 32 * b);
      }
    }
  }

  __device__ __forceinline__ void take_q(const KvAttnArgs& a, int j, const Fetched& fetched) {
    float x[NB][8];
    uint32_t top = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (E == 0) {
          x[b][i] = __builtin_bit_cast(float, uint32_t(fetched.w[b][0][i]));
          x[b][4 + i] = __builtin_bit_cast(float, uint32_t(fetched.w[b][E == 0][i]));
        } else {
          const uint32_t bits = fetched.w[b][0][i];
          x[b][2 * i] = unpack16<E == 1>(bits & 0xFFFFu);
          x[b][2 * i + 1] = unpack16<E == 1>(bits >> 16);
        }
      }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, x[b][i]) & 0x7FFFFFFFu);
    top = over_column(top, [](uint32_t a, uint32_t b) { return max(a, b); });
    // 2^up brings the largest value to [2^14, 2^15); up to 2^126 for f32 that are next to nothing
    const int up = min(126, 14 - (int(top >> 23) - 127));
    const float scale = __builtin_copysignf(__builtin_bit_cast(float, uint32_t(127 + up) << 23), a.scale);
    factor[j] = top >= 0x7F800000u ? __builtin_nanf("") : fabsf(a.scale) * __builtin_bit_cast(float, uint32_t(127 - up) << 23);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = x[b][2 * i] * scale, z = x[b][2 * i + 1] * scale;
        const uint32_t w = pack16<true>(y, z);
        q[j][b][0][i] = w;
        if constexpr (QP == 2) q[j][b][1][i] = pack16<true>(y - unpack16<true>(w & 0xFFFFu), z - unpack16<true>(w >> 16));
      }
    }
  }

  // 32 tokens from position `at`; MASK: some row may not see all of them; there0, there1: the
  // page of the first, second 16 is there.  T gives the operands k(i, b), v(b, m) and the scales
  // ks(i, b), vs(i, b).
  template <bool MASK, class T>
  __device__ __forceinline__ void step(const T& t, int at, bool there0, bool there1, int lane) {
    const int quad = lane >> 4;
    f32x4 s[TILES][2];
    bool seen[TILES][2][4];
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) s[j][i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4 k = t.k(i, b);
        const u32x2 ks = t.ks(i, b);
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          f32x4 d = mfma16<true>(k, q[j][b][0], f32x4{0, 0, 0, 0});
          if constexpr (QP == 2) d = mfma16<true>(k, q[j][b][1], d);
#pragma unroll
          for (int r = 0; r < 4; ++r) s[j][i][r] = fmaf(d[r], half_of(ks, r), s[j][i][r]);
        }
      }
    u32x2 vs[2][NB];
    uint32_t top_scale = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        vs[i][b] = t.vs(i, b);
        if constexpr (!MASK) top_scale = max_u16(top_scale, max_u16(vs[i][b][0] & 0x7FFF7FFFu, vs[i][b][1] & 0x7FFF7FFFu));
      }
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      uint32_t top_v = top_scale;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s[j][i][r] *= factor[j];
          if constexpr (MASK) {
            const int p = at + 16 * i + 4 * quad + r;
            seen[j][i][r] = (i ? there1 : there0) && p >= lo[j] && p < hi[j];
            s[j][i][r] = seen[j][i][r] ? s[j][i][r] : -kInf;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const uint32_t w = vs[i][b][r >> 1];
              top_v = max(top_v, seen[j][i][r] ? w >> (16 * (r & 1)) & 0x7FFFu : 0u);
            }
          }
        }
      if constexpr (!MASK) top_v = max(top_v & 0xFFFFu, top_v >> 16);
      float most = s[j][0][0];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) most = fmaxf(most, s[j][i][r]);
      most += float(int(top_v >> 10 & 31u) - 14);  // V's scales lie below 2^(exponent - 14)
      if (__builtin_expect(__any(most > ref[j] + 15.0f), 0)) raise(j, most);
      const float from = ref[j] == -kInf ? 0.0f : ref[j];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s[j][i][r] = __builtin_amdgcn_exp2f(s[j][i][r] - from);
          sum[j] += s[j][i][r];
        }
    }
    // s is p now; what a row does not see is zero, whatever its scale
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const u32x4 v0 = t.v(b, 0), v1 = t.v(b, 1);
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        float pv[8];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float sv = half_of(vs[i][b], r);
            if constexpr (MASK) sv = seen[j][i][r] ? sv : 0.0f;
            pv[4 * i + r] = s[j][i][r] * sv;
          }
        u32x4 p, pl;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = pack16<true>(pv[2 * i], pv[2 * i + 1]);
          p[i] = w;
          if constexpr (PP == 2)
            pl[i] = pack16<true>(pv[2 * i] - unpack16<true>(w & 0xFFFFu), pv[2 * i + 1] - unpack16<true>(w >> 16));
        }
        o[j][b][0] = mfma16<true>(v0, p, o[j][b][0]);
        o[j][b][1] = mfma16<true>(v1, p, o[j][b][1]);
        if constexpr (PP == 2) {
          o[j][b][0] = mfma16<true>(v0, pl, o[j][b][0]);
          o[j][b][1] = mfma16<true>(v1, pl, o[j][b][1]);
        }
      }
    }
  }
  // The same with operands that have their scales in them: K 2^up_k and V 2^up_v, both below 2^15, in f16
  // (bf16 calls) or as two f16 parts, without the product of two low parts.  The probabilities enter
  // as p 2^-up_v, which the reference keeps below 2^15 as above.
  template <bool MASK, class T>
  __device__ __forceinline__ void fold_step(const T& t, int at, bool there0, bool there1, int up_k0, int up_k1, int up_v,
                                            int lane) {
    const int quad = lane >> 4;
    const float up = __builtin_bit_cast(float, uint32_t(127 + up_v) << 23);
    f32x4 s[TILES][2];
    // operands of the next group of blocks are on their way from LDS while the products of one run
    constexpr int G = PP == 2 ? 1 : 2, kGroups = (NB + G - 1) / G;
    u32x4 hold[2][G][2][PP];
    auto load_k = [&](int g) {
#pragma unroll
      for (int c = 0; c < G; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (g * G + c < NB) {
            hold[g & 1][c][i][0] = t.k(i, g * G + c);
            if constexpr (PP == 2) hold[g & 1][c][i][1] = t.k_low(i, g * G + c);
          }
    };
    auto load_v = [&](int g) {
#pragma unroll
      for (int c = 0; c < G; ++c)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          if (g * G + c < NB) {
            hold[g & 1][c][m][0] = t.v(g * G + c, m);
            if constexpr (PP == 2) hold[g & 1][c][m][1] = t.v_low(g * G + c, m);
          }
    };
    load_k(0);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (g + 1 < kGroups) load_k(g + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int part = 0; part < PP + QP - 1; ++part)  // K q, then K's low part, or q's
#pragma unroll
        for (int c = 0; c < G; ++c) {
          const int b = g * G + c;
          if (b >= NB) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < TILES; ++j)
              s[j][i] = mfma16<true>(hold[g & 1][c][i][part == 1], q[j][b][part == 2], b || part ? s[j][i] : f32x4{0, 0, 0, 0});
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    load_v(0);
    u32x4 p[TILES], pl[TILES];
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      bool seen[2][4];
      float top[2], f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = -kInf;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (MASK) {
            const int pos = at + 16 * i + 4 * quad + r;
            seen[i][r] = (i ? there1 : there0) && pos >= lo[j] && pos < hi[j];
            top[i] = fmaxf(top[i], seen[i][r] ? s[j][i][r] : -kInf);
          } else {
            top[i] = fmaxf(top[i], s[j][i][r]);
          }
        }
        f[i] = factor[j] * __builtin_bit_cast(float, uint32_t(127 - (i ? up_k1 : up_k0)) << 23);
      }
      const float most = fmaxf(top[0] * f[0], top[1] * f[1]) - float(up_v);
      if (__builtin_expect(__any(most > ref[j] + 15.0f), 0)) raise(j, most);
      const float from = (ref[j] == -kInf ? 0.0f : ref[j]) + float(up_v);
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = __builtin_amdgcn_exp2f(fmaf(s[j][i][r], f[i], -from));
          if constexpr (MASK) x = seen[i][r] ? x : 0.0f;
          s[j][i][r] = x;
          part += x;
        }
      sum[j] = fmaf(part, up, sum[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = s[j][i >> 1][2 * (i & 1)], y = s[j][i >> 1][2 * (i & 1) + 1];
        const uint32_t w = pack16<true>(x, y);
        p[j][i] = w;
        if constexpr (PP == 2) pl[j][i] = pack16<true>(x - unpack16<true>(w & 0xFFFFu), y - unpack16<true>(w >> 16));
      }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (g + 1 < kGroups) load_v(g + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int part = 0; part < 2 * PP - 1; ++part)  // V p, then V's low part, then p's
#pragma unroll
        for (int c = 0; c < G; ++c) {
          const int b = g * G + c;
          if (b >= NB) continue;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < TILES; ++j)
              o[j][b][m] = mfma16<true>(hold[g & 1][c][m][part == 1], part == 2 ? pl[j] : p[j], o[j][b][m]);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // A new reference for the columns in which products could pass 2^15: they start at 2^7 again.
  __device__ __forceinline__ void raise(int j, float most) {
    const float need = column_max(most);
    const float next = need > ref[j] + 15.0f ? need - 7.0f : ref[j];
    const float f = ref[j] == -kInf ? 0.0f : __builtin_amdgcn_exp2f(ref[j] - next);
    ref[j] = next;
    sum[j] *= f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[j][b][m][r] *= f;
  }
  template <class T>
  __device__ __forceinline__ void work(const T& t, int at, bool there0, bool there1, int lane) {
    if (there0 && there1 && at >= all_lo && at + 32 <= all_hi) step<false>(t, at, true, true, lane);
    else step<true>(t, at, there0, there1, lane);
  }

  // A tile's result, its sum already that of the whole column: final, or a part for the join.
  __device__ __forceinline__ void store(const KvAttnArgs& a, int j, const Row& row, int slot, int lane) {
    if (row.token < 0) return;
    const int64_t at = row.token * int64_t(a.q_heads) + row.head;
    if (a.slots) {
      const int64_t part = at * a.slots + slot;
      if (lane < 16) a.stats[part] = make_float2(ref[j], sum[j]);
      if (sum[j] != 0.0f) {  // nothing seen: the join does not look at it
#pragma unroll
        for (int i = 0; i < NB * 2; ++i)
          *reinterpret_cast<f32x4*>(a.sums + part * (32 * NB) + 16 * i + 4 * (lane >> 4)) = o[j][i >> 1][i & 1];
      }
      return;
    }
    const float inv = 1.0f / sum[j];
    if (a.lse && lane < 16)
      a.lse[at] = sum[j] == 0.0f ? -kInf : 0.69314718f * (ref[j] + __builtin_amdgcn_logf(sum[j]));
    const int64_t to = row.token * a.out_token + row.head * a.out_head + 4 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < NB * 2; ++i) {
      f32x4 v = o[j][i >> 1][i & 1] * inv;
      if (sum[j] == 0.0f) v = f32x4{0, 0, 0, 0};
      if constexpr (E == 0) {
        __builtin_memcpy(static_cast<float*>(a.out) + to + 16 * i, &v, 16);
      } else {
        const u32x2 x = {pack16<E == 1>(v[0], v[1]), pack16<E == 1>(v[2], v[3])};
        __builtin_memcpy(static_cast<uint16_t*>(a.out) + to + 16 * i, &x, 8);
      }
    }
  }
};

// Two sets in LDS as they are in the cache, and their codes as f16 operands.
template <bool Q4, int NB>
struct Raw {
  static constexpr int C = Q4 ? 256 : 512, kSet = NB * (2 * C + 64), kPieces = kSet / 16;
  static constexpr int W = Q4 ? 1 : 2;  // words of a lane and block
  const u32x4* at;                      // kPieces each
  int lane;

  __device__ __forceinline__ const uint8_t* bytes(int i) const { return reinterpret_cast<const uint8_t*>(at + i * kPieces); }
  // of K's block b: the lane's token, 8 dimensions
  __device__ __forceinline__ u32x4 k(int i, int b) const {
    uint32_t w[W];
    __builtin_memcpy(w, __builtin_assume_aligned(bytes(i) + b * C + lane * (4 * W), 4 * W), 4 * W);
    if constexpr (Q4) {
      const uint32_t lo = w[0] & 0x0F0F0F0Fu, hi = w[0] >> 4 & 0x0F0F0F0Fu;
      return u32x4{codes16<8>(lo, 0x04010400u), codes16<8>(lo, 0x04030402u), codes16<8>(hi, 0x04010400u),
                   codes16<8>(hi, 0x04030402u)};
    } else {
      return u32x4{codes16<128>(w[0], 0x04010400u), codes16<128>(w[0], 0x04030402u), codes16<128>(w[1], 0x04010400u),
                   codes16<128>(w[1], 0x04030402u)};
    }
  }
  // of V's block b, dimensions 16 m .. 16 m + 15: the lane's dimension, 4 + 4 tokens
  __device__ __forceinline__ u32x4 v(int b, int m) const {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t x[W];
      __builtin_memcpy(x, __builtin_assume_aligned(bytes(i) + (NB + b) * C + lane * (4 * W), 4 * W), 4 * W);
      if constexpr (Q4) w[i] = x[0] >> (4 * m) & 0x0F0F0F0Fu;
      else w[i] = x[m];
    }
    constexpr int BIAS = Q4 ? 8 : 128;
    return u32x4{codes16<BIAS>(w[0], 0x04010400u), codes16<BIAS>(w[0], 0x04030402u), codes16<BIAS>(w[1], 0x04010400u),
                 codes16<BIAS>(w[1], 0x04030402u)};
  }
  __device__ __forceinline__ u32x2 scales(int i, int plane, int b) const {
    return *reinterpret_cast<const u32x2*>(bytes(i) + NB * (2 * C + 32 * plane) + ((lane >> 4) * NB + b) * 8);
  }
  __device__ __forceinline__ u32x2 ks(int i, int b) const { return scales(i, 0, b); }
  __device__ __forceinline__ u32x2 vs(int i, int b) const { return scales(i, 1, b); }

  // Starts copies of set `set` of page `page` (0 for one that is not there) to dst: kCopies of them.
  static constexpr int kCopies = (kPieces + 63) / 64;
  static __device__ __forceinline__ void copy(const KvArgs& a, int head, int page, int set, u32x4* dst, int lane) {
    const Buf src = buffer_of(a.data + max(page, 0) * a.page_bytes + int64_t(head) * a.head_bytes + set * a.set_bytes);
#pragma unroll
    for (int c = 0; c < kPieces / 64; ++c) copy_to_lds(src, lane * 16, c * 1024, dst + c * 64);
    if constexpr (kPieces % 64 != 0)
      if (lane < kPieces % 64) copy_to_lds(src, lane * 16, kPieces / 64 * 1024, dst + kPieces / 64 * 64);
  }
};

// Pages of the next 32 steps: lane 2 n + i holds the page and place of set i of step n.
struct Ahead {
  int pages, places;
  // step n: sets first + stride n and the next, up to end
  __device__ __forceinline__ void look_up(const KvArgs& kv, const int32_t* table, int first, int stride, int n0, int end,
                                          int lane) {
    const int64_t u = first + int64_t(stride) * (n0 + (lane >> 1)) + (lane & 1);
    int set, page = -1;
    const int p = kv_page_of(kv, uint32_t(min(u, int64_t(end - 1))), set);
    if (u < end) {
      page = table[p];
      if (page < 0 || page >= kv.pages) page = -1;
    }
    pages = page;
    places = set;
  }
  __device__ __forceinline__ int page(int n, int i) const { return __builtin_amdgcn_readlane(pages, 2 * (n & 31) + i); }
  __device__ __forceinline__ int place(int n, int i) const { return __builtin_amdgcn_readlane(places, 2 * (n & 31) + i); }
};

template <int N>
__device__ __forceinline__ void wait_copies() {  // until at most N are under way
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// What this wave has read of LDS has arrived: copies may overwrite it.
__device__ __forceinline__ void lds_read() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Blocks of 16 queries, of a sequence that has up to 64 of a head: every wave has tokens of
// its own, 32 of them under way to its part of LDS while it works on 32 others; no barrier
// before the waves meet.  Bound by
// memory where there are many tokens: 64 ragged sequences of up to 16000 (444000 in all, 32 / 8 heads of 128,
// Q8_0, bf16) take 192 us, 5.0 TB/s.  4-bit codes cost more instructions a byte: 96 sequences of up to 1000
// tokens of their own behind a prefix (Q4_0, f16) take 30 us, 1.9 TB/s; three workgroups a unit, where
// they fit, instead of two: 33 -> 30.
// grid: (k / v heads * splits * sequences (1 for the prefix), row blocks)
template <bool Q4, int E, int NB, bool PREFIX>
__global__ __launch_bounds__(256, Q4 && NB <= 4 ? 3 : 2) void kv_attention_few_kernel(const KvAttnArgs a, int splits,
                                                                                      int first_slot) {
  typedef Raw<Q4, NB> R;
  constexpr int kStep = 2 * R::kPieces, kMeet = 3 * NB * 2 * 64;  // 16-byte pieces
  __shared__ u32x4 ring0[kStep * 4 > kMeet ? kStep * 4 : kMeet], ring1[kStep * 4];
  __shared__ float2 meet_stats[3][64];
  const KvArgs& kv = a.kv;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Span sp = span_of<PREFIX>(a, splits);
  for (uint32_t base = blockIdx.y * 16; base < sp.rows; base += gridDim.y * 16) {
    Sequences seq;
    if constexpr (PREFIX) seq.look_up(kv, int(base / uint32_t(a.group)), lane);
    Row row[1] = {row_of<PREFIX>(a, seq, base + (lane & 15), sp.rows, sp.kv_head, sp.r0, sp.first_pos, PREFIX ? 0 : a.prefix,
                                 sp.cap)};
    typedef Rows<E, NB, 1> Wave;
    Wave w;
    typename Wave::Fetched q;
    Wave::fetch_q(a, row[0], lane, q);
    w.begin(row);
    int u0, u1;
    share_of(w.any_lo >> 4, (w.any_hi + 15) >> 4, splits, sp.split, 8, kLeastFew, u0, u1);
    const int first = u0 + 2 * wave, steps = u1 > first ? (u1 - first + 7) >> 3 : 0;  // sets first + 8 n and the next
    Ahead ahead;
    auto fetch = [&](u32x4* ring, int n) {
      lds_read();
      if ((n & 31) == 0) ahead.look_up(kv, sp.table, first, 8, n, u1, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        R::copy(kv, sp.kv_head, ahead.page(n, i), ahead.place(n, i), ring + wave * kStep + i * R::kPieces, lane);
    };
    if (steps > 0) {
      fetch(ring0, 0);
      w.take_q(a, 0, q);
      bool a0 = ahead.page(0, 0) >= 0, a1 = ahead.page(0, 1) >= 0;
      for (int n = 0; n < steps; n += 2) {
        bool b0 = false, b1 = false;
        if (n + 1 < steps) {
          fetch(ring1, n + 1);
          b0 = ahead.page(n + 1, 0) >= 0, b1 = ahead.page(n + 1, 1) >= 0;
          wait_copies<2 * R::kCopies>();
        } else {
          wait_copies<0>();
        }
        w.work(R{ring0 + wave * kStep, lane}, (first + 8 * n) * 16, a0, a1, lane);
        if (n + 1 >= steps) break;
        if (n + 2 < steps) {
          fetch(ring0, n + 2);
          a0 = ahead.page(n + 2, 0) >= 0, a1 = ahead.page(n + 2, 1) >= 0;
          wait_copies<2 * R::kCopies>();
        } else {
          wait_copies<0>();
        }
        w.work(R{ring1 + wave * kStep, lane}, (first + 8 * (n + 1)) * 16, b0, b1, lane);
      }
    }

    // the four waves meet: the first adds the others' results to its own
    w.sum[0] = column_sum(w.sum[0]);
    f32x4* meet = reinterpret_cast<f32x4*>(ring0);
    __syncthreads();
    if (wave) {
#pragma unroll
      for (int i = 0; i < NB * 2; ++i) meet[((wave - 1) * NB * 2 + i) * 64 + lane] = w.o[0][i >> 1][i & 1];
      meet_stats[wave - 1][lane] = make_float2(w.ref[0], w.sum[0]);
    }
    __syncthreads();
    if (!wave) {
      float ref = w.ref[0];
#pragma unroll
      for (int k = 0; k < 3; ++k) ref = fmaxf(ref, meet_stats[k][lane].x);
      const float from = ref == -kInf ? 0.0f : ref, f = __builtin_amdgcn_exp2f(w.ref[0] - from);
      w.ref[0] = ref;
      w.sum[0] *= f;
#pragma unroll
      for (int i = 0; i < NB * 2; ++i) w.o[0][i >> 1][i & 1] *= f;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const float2 st = meet_stats[k][lane];
        const float g = __builtin_amdgcn_exp2f(st.x - from);
        w.sum[0] = fmaf(st.y, g, w.sum[0]);
#pragma unroll
        for (int i = 0; i < NB * 2; ++i) {
          const f32x4 v = meet[(k * NB * 2 + i) * 64 + lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) w.o[0][i >> 1][i & 1][r] = fmaf(v[r], g, w.o[0][i >> 1][i & 1][r]);
        }
      }
      w.store(a, 0, row[0], first_slot + sp.split, lane);
    }
    __syncthreads();  // the next rows' tokens go where the results were
  }
}

// A step's operands in LDS, made once for the four waves: K and V with their scales, in PARTS
// f16 parts.
template <int NB, int PARTS>
struct Ready {
  u32x4 kc[PARTS][2][NB][64], vc[PARTS][NB][2][64];
  int up_k[2], up_v;  // of K's sets
};
template <int NB, int PARTS>
struct ReadyView {
  const Ready<NB, PARTS>* r;
  int lane;
  __device__ __forceinline__ u32x4 k(int i, int b) const { return r->kc[0][i][b][lane]; }
  __device__ __forceinline__ u32x4 v(int b, int m) const { return r->vc[0][b][m][lane]; }
  __device__ __forceinline__ u32x4 k_low(int i, int b) const { return r->kc[PARTS - 1][i][b][lane]; }
  __device__ __forceinline__ u32x4 v_low(int b, int m) const { return r->vc[PARTS - 1][b][m][lane]; }
};

__device__ __forceinline__ uint32_t pk_mul(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) * __builtin_bit_cast(f16x2, b));
}
// Codes times scales: rounded to f16, and what the rounding left over (exact: the product has 19 bits).
template <int PARTS>
__device__ __forceinline__ void put_scaled(u32x4 codes, u32x4 scales, u32x4* hi, u32x4* low) {
  u32x4 h, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = codes[i], s = scales[i], w = pk_mul(c, s);
    h[i] = w;
    if constexpr (PARTS == 2)
      l[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, c), __builtin_bit_cast(f16x2, s),
                                                                    -__builtin_bit_cast(f16x2, w)));
  }
  *hi = h;
  if constexpr (PARTS == 2) *low = l;
}

// Exponent that brings scales below 2^(e - 14), e their largest biased exponent, below 2^8: with codes up to
// 128 that is 2^15.  2^up is an f16 value.
__device__ __forceinline__ int up_of(uint32_t top) { return min(15, 22 - int(top >> 10)); }
__device__ __forceinline__ uint32_t two_to(int up) { return uint32_t(15 + up) << 10; }

// A wave's share of a step's operands: a set of K, or half of V's dimensions; with eight waves
// half of the blocks of those.
// Scales of positions outside lo .. hi - 1, which no row sees, are zeros in V (a probability of zero times
// whatever lies there is zero then).  A scale that is no number makes its token's scores NaN, V's too, and
// is zero in V.
template <int WAVES, bool Q4, int NB, int PARTS>
__device__ __forceinline__ void make_ready(const Raw<Q4, NB>& raw, Ready<NB, PARTS>& to, int wave, int at, int lo, int hi,
                                           int there) {
  constexpr int C = Raw<Q4, NB>::C;
  const int lane = raw.lane, share = wave >> 2;
  auto mine = [&](int b) { return WAVES == 4 || (b >= (NB + 1) / 2) == (share != 0); };
  if ((wave & 3) < 2) {
    const int i = wave & 1, ln = lane & 15, p = at + 16 * i + ln;
    const uint16_t* sc = reinterpret_cast<const uint16_t*>(raw.bytes(i) + 2 * NB * C) + (ln >> 2) * NB * 4 + (ln & 3);
    uint32_t s[NB], top = 0, worst = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      s[b] = sc[4 * b];
      worst = max(worst, uint32_t(sc[16 * NB + 4 * b]) & 0x7FFFu);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t half = s[b] & 0x7FFFu;
      top = max(top, half < 0x7C00u ? half : 0u);
    }
    top = uint32_t(row_max((there >> i & 1) && p >= lo && p < hi ? int(top) : 0));  // the four rows hold the same tokens
    const int up = up_of(uint32_t(__builtin_amdgcn_readfirstlane(int(top))));
    if (worst >= 0x7C00u) s[0] = 0x7E00u;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (!mine(b)) continue;
      const uint32_t x = pk_mul(s[b] * 0x10001u, two_to(up) * 0x10001u);
      put_scaled<PARTS>(raw.k(i, b), u32x4{x, x, x, x}, &to.kc[0][i][b][lane], &to.kc[PARTS - 1][i][b][lane]);
    }
    if (!share && lane == 0) to.up_k[i] = up;
  } else {
    const int m = wave & 1;
    u32x2 s[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) s[b][i] = raw.vs(i, b);
    if (there != 3 || at < lo || at + 32 > hi) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = at + 16 * i + 4 * (lane >> 4) + 2 * h;
          const uint32_t keep = (p >= lo && p < hi ? 0xFFFFu : 0u) | (p + 1 >= lo && p + 1 < hi ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int b = 0; b < NB; ++b) s[b][i][h] &= there >> i & 1 ? keep : 0u;
        }
    }
    auto top_of = [&]() -> uint32_t {
      uint32_t top = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) top = max_u16(top, max_u16(s[b][i][0] & 0x7FFF7FFFu, s[b][i][1] & 0x7FFF7FFFu));
      top = over_column(top, [](uint32_t a, uint32_t b) { return max_u16(a, b); });
      return uint32_t(__builtin_amdgcn_readfirstlane(int(max(top & 0xFFFFu, top >> 16))));
    };
    uint32_t top = top_of();
    if (__builtin_expect(top >= 0x7C00u, 0)) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w = s[b][i][h];
            s[b][i][h] = ((w & 0x7FFFu) < 0x7C00u ? w & 0xFFFFu : 0u) | ((w >> 16 & 0x7FFFu) < 0x7C00u ? w & 0xFFFF0000u : 0u);
          }
      top = top_of();
    }
    const int up = up_of(top);
    const uint32_t by = two_to(up) * 0x10001u;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (!mine(b)) continue;
      const u32x4 x = {pk_mul(s[b][0][0], by), pk_mul(s[b][0][1], by), pk_mul(s[b][1][0], by), pk_mul(s[b][1][1], by)};
      put_scaled<PARTS>(raw.v(b, m), x, &to.vc[0][b][m][lane], &to.vc[PARTS - 1][b][m][lane]);
    }
    if (m == 0 && !share && lane == 0) to.up_v = up;
  }
}
// Many queries: each of the four or eight waves has 16 * TILES rows of its own and all work on the
// same 32 tokens.  A step's bytes are copied to LDS two steps ahead and made into operands, a
// quarter by each wave, one step ahead, so that a step has one barrier and its vector and
// matrix instructions come from different steps.  Operands leave LDS a group of blocks ahead of
// their products.  Bound by vector and matrix instructions in turn (a prefix of 8200 tokens for 384 rows of
// each of 8 heads of 128, Q4_0, f16: 57 us, of which the steps 37: 2900 clocks for 128 rows and 32 tokens
// against 1280 of matrix instructions, five products for the definition's two; a chunk of 700 tokens
// with a window of 1500, 14 / 2 heads of 96, Q8_0, bf16: 30 us, of which the steps 14).
// Where two workgroups of a unit would not fit its LDS with two steps of bytes (or one
// with more than 128 dimensions), the next bytes are copied behind a second barrier.
template <bool Q4, int E, int NB, int WAVES, int TILES, bool PREFIX>
__global__ __launch_bounds__(64 * WAVES, 2) void kv_attention_many_kernel(const KvAttnArgs a, int splits, int first_slot) {
  typedef Raw<Q4, NB> R;
  constexpr int kStep = 2 * R::kPieces, kRows = 16 * TILES * WAVES;
  constexpr int kParts = Rows<E, NB, TILES>::PP;
  constexpr size_t kRoom = (NB > 4 ? 160 : 80) * 1024 - 64;
  constexpr bool kTwoRaws = 2 * sizeof(Ready<NB, kParts>) + 32 * kStep <= kRoom;
  static_assert(2 * sizeof(Ready<NB, kParts>) + 16 * kStep <= kRoom);
  __shared__ u32x4 raws[kTwoRaws ? 2 : 1][kStep];
  __shared__ Ready<NB, kParts> ready0, ready1;
  __shared__ int range[WAVES][2];
  const KvArgs& kv = a.kv;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Span sp = span_of<PREFIX>(a, splits);
  for (uint32_t base = blockIdx.y * kRows; base < sp.rows; base += gridDim.y * kRows) {
    Row row[TILES];
    Sequences seq;
    if constexpr (PREFIX) seq.look_up(kv, int(min(base + wave * (16 * TILES), sp.rows - 1) / uint32_t(a.group)), lane);
#pragma unroll
    for (int j = 0; j < TILES; ++j)
      row[j] = row_of<PREFIX>(a, seq, base + wave * (16 * TILES) + 16 * j + (lane & 15), sp.rows, sp.kv_head, sp.r0,
                              sp.first_pos, PREFIX ? 0 : a.prefix, sp.cap);
    typedef Rows<E, NB, TILES> Wave;
    Wave w;
    typename Wave::Fetched q[TILES];
#pragma unroll
    for (int j = 0; j < TILES; ++j) Wave::fetch_q(a, row[j], lane, q[j]);
    w.begin(row);
    if (lane == 0) range[wave][0] = w.any_lo < w.any_hi ? w.any_lo : 0x7FFFFFFF, range[wave][1] = w.any_hi;
    lds_barrier16();
    int lo = range[0][0], hi = range[0][1];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) lo = min(lo, range[i][0]), hi = max(hi, range[i][1]);
    lo = __builtin_amdgcn_readfirstlane(lo), hi = __builtin_amdgcn_readfirstlane(hi);
    int u0, u1;
    share_of(lo < hi ? lo >> 4 : 0, lo < hi ? (hi + 15) >> 4 : 0, splits, sp.split, 2, kLeastMany, u0, u1);
    const int steps = u1 > u0 ? (u1 - u0 + 1) >> 1 : 0;
    Ahead ahead;
    // half of the waves copy a set, a part each; returns which sets are there, as bits
    auto fetch = [&](u32x4* raw, int n) -> int {
      if ((n & 31) == 0) ahead.look_up(kv, sp.table, u0, 2, n, u1, lane);
      const int i = wave / (WAVES / 2), part = wave % (WAVES / 2), p0 = ahead.page(n, 0), p1 = ahead.page(n, 1);
      const int both = int(p0 >= 0) | int(p1 >= 0) << 1;
      const Buf src = buffer_of(kv.data + max(i ? p1 : p0, 0) * kv.page_bytes + int64_t(sp.kv_head) * kv.head_bytes +
                                (i ? ahead.place(n, 1) : ahead.place(n, 0)) * kv.set_bytes);
      constexpr int kPart = R::kPieces / (WAVES / 2);
      static_assert(kPart * (WAVES / 2) == R::kPieces);
      u32x4* dst = raw + i * R::kPieces + part * kPart;
#pragma unroll
      for (int c = 0; c < kPart / 64; ++c) copy_to_lds(src, lane * 16, (part * kPart + c * 64) * 16, dst + c * 64);
      if constexpr (kPart % 64 != 0)
        if (lane < kPart % 64) copy_to_lds(src, lane * 16, (part * kPart + kPart / 64 * 64) * 16, dst + kPart / 64 * 64);
      return both;
    };
    u32x4 *const raw0 = raws[0], *const raw1 = raws[kTwoRaws ? 1 : 0];
    int there = 0, there1 = 0, there2 = 0;  // of step n and the next two
    auto turn = [&](u32x4* raw, const u32x4* raw_next, const Ready<NB, kParts>& ready, Ready<NB, kParts>& ready_next, int n) {
      wait_copies<0>();
      lds_barrier16();  // step n is ready, n + 1 has landed; nobody works on step n - 1 any more
      const int at = (u0 + 2 * n) * 16;
      if (kTwoRaws && n + 2 < steps) there2 = fetch(raw, n + 2);
      if (n + 1 < steps) make_ready<WAVES>(R{raw_next, lane}, ready_next, wave, at + 32, lo, hi, there1);
      if constexpr (!kTwoRaws) {
        if (n + 2 < steps) {
          lds_barrier16();
          there2 = fetch(raw, n + 2);
        }
      }
      if (at < w.any_hi && at + 32 > w.any_lo) {
        const ReadyView<NB, kParts> view{&ready, lane};
        const int k0 = __builtin_amdgcn_readfirstlane(ready.up_k[0]), k1 = __builtin_amdgcn_readfirstlane(ready.up_k[1]);
        const int v = __builtin_amdgcn_readfirstlane(ready.up_v);
        if (there == 3 && at >= w.all_lo && at + 32 <= w.all_hi)
          w.template fold_step<false>(view, at, true, true, k0, k1, v, lane);
        else
          w.template fold_step<true>(view, at, there & 1, there & 2, k0, k1, v, lane);
      }
      there = there1, there1 = there2;
    };
    if (steps > 0) {
      there = fetch(raw0, 0);
      if (kTwoRaws && steps > 1) there1 = fetch(raw1, 1);
#pragma unroll
      for (int j = 0; j < TILES; ++j) w.take_q(a, j, q[j]);
      wait_copies<0>();
      lds_barrier16();
      make_ready<WAVES>(R{raw0, lane}, ready0, wave, u0 * 16, lo, hi, there);
      if constexpr (!kTwoRaws) {
        if (steps > 1) {
          lds_barrier16();
          there1 = fetch(raw1, 1);
        }
      }
      for (int n = 0; n < steps; n += 2) {
        turn(raw0, raw1, ready0, ready1, n);
        if (n + 1 < steps) turn(raw1, raw0, ready1, ready0, n + 1);
      }
    }
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      w.sum[j] = column_sum(w.sum[j]);
      w.store(a, j, row[j], first_slot + sp.split, lane);
    }
    __syncthreads();  // range, and the steps' buffers, are done with
  }
}

}  // namespace

constexpr int kManyRows = 128;  // of a workgroup of the kernel for many

// One head size's launches.
template <bool Q4, int E, int NB>
hipError_t kv_attention_go(const KvAttnArgs& a, const KvAttentionPlan& p, hipStream_t s) {
  const unsigned heads = unsigned(a.kv.heads);
  // 128 rows of heads of more than 128 values: eight waves of one tile, as four of two would need all registers of
  // their unit (a chunk of 700 tokens of 16 heads over 6000, Q8_0: bf16, 256 values 240 -> 203 us, f16, 160 values 224 -> 178)
  constexpr int W = NB > 4 ? 8 : 4, T = kManyRows / (16 * W);
  constexpr unsigned kMany = 64 * W;
  if (a.prefix) {
    const dim3 grid(heads * unsigned(p.prefix_splits), unsigned(p.prefix_row_blocks), 1);
    const int n = p.prefix_splits;
    if (p.prefix_many) hipLaunchKernelGGL((kv_attention_many_kernel<Q4, E, NB, W, T, true>), grid, dim3(kMany), 0, s, a, n, 0);
    else hipLaunchKernelGGL((kv_attention_few_kernel<Q4, E, NB, true>), grid, dim3(256), 0, s, a, n, 0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int first = a.prefix ? p.prefix_splits : 0, n = p.splits;
  const dim3 grid(heads * unsigned(p.splits) * unsigned(a.kv.B), unsigned(p.row_blocks), 1);
  if (p.many) hipLaunchKernelGGL((kv_attention_many_kernel<Q4, E, NB, W, T, false>), grid, dim3(kMany), 0, s, a, n, first);
  else hipLaunchKernelGGL((kv_attention_few_kernel<Q4, E, NB, false>), grid, dim3(256), 0, s, a, n, first);
  return hipGetLastError();
}

template <bool Q4, int E>
hipError_t kv_attention_sizes(const KvAttnArgs& a, const KvAttentionPlan& p, hipStream_t s) {
  switch (a.kv.nb) {
    case 1: return kv_attention_go<Q4, E, 1>(a, p, s);
    case 2: return kv_attention_go<Q4, E, 2>(a, p, s);
    case 3: return kv_attention_go<Q4, E, 3>(a, p, s);
    case 4: return kv_attention_go<Q4, E, 4>(a, p, s);
    case 5: return kv_attention_go<Q4, E, 5>(a, p, s);
    case 6: return kv_attention_go<Q4, E, 6>(a, p, s);
    case 7: return kv_attention_go<Q4, E, 7>(a, p, s);
    default: return kv_attention_go<Q4, E, 8>(a, p, s);
  }
}

// kv_attention_{q8,q4}_{f32,f16,bf16}.hip
hipError_t kv_attention_q8_f32(const KvAttnArgs&, const KvAttentionPlan&, hipStream_t);
hipError_t kv_attention_q8_f16(const KvAttnArgs&, const KvAttentionPlan&, hipStream_t);
hipError_t kv_attention_q8_bf16(const KvAttnArgs&, const KvAttentionPlan&, hipStream_t);
hipError_t kv_attention_q4_f32(const KvAttnArgs&, const KvAttentionPlan&, hipStream_t);
hipError_t kv_attention_q4_f16(const KvAttnArgs&, const KvAttentionPlan&, hipStream_t);
hipError_t kv_attention_q4_bf16(const KvAttnArgs&, const KvAttentionPlan&, hipStream_t);

}  // namespace qmv
