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
// Largest value of the wave, in every lane.
__device__ __forceinline__ int wave_max(int v) {
  v = max(v, dpp_of<0xB1>(v));
  v = max(v, dpp_of<0x4E>(v));
  v = max(v, dpp_of<0x141>(v));
  v = max(v, dpp_of<0x140>(v));
  v = max(v, __shfl_xor(v, 16));
  return __builtin_amdgcn_readfirstlane(max(v, __shfl_xor(v, 32)));
}
// Over the four lanes of a column (lane ^ 16, lane ^ 32).
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
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

// Where q rows of this launch's tile lie.  A row r of a sequence (or, for the shared
// prefix, of the whole call) is token r / group and head r % group of the k / v head.
struct Row {
  int token;   // row of q, -1: none
  int lo, hi;  // positions that it sees
};

template <bool Q4, int E, int NB>
struct Step {  // 32 tokens: two sets of 16 in the lane's share
  static constexpr int W = Q4 ? 1 : 2;  // words of a lane and block
  uint32_t k[2][NB][W], v[2][NB][W];
  uint32_t ks[2][NB][2], vs[2][NB][2];  // four tokens' scales
  bool there[2];

  __device__ __forceinline__ void load(const KvArgs& a, int head, int i, int page, int set, int lane) {
    constexpr int C = Q4 ? 256 : 512;
    there[i] = page >= 0;
    const uint8_t* p = a.data + max(page, 0) * a.page_bytes + int64_t(head) * a.head_bytes + set * a.set_bytes;
    const uint32_t code_at = uint32_t(lane) * (4 * W), scale_at = uint32_t(lane >> 4) * (8 * NB);
#pragma unroll
    for (int b = 0; b < NB; ++b) __builtin_memcpy(k[i][b], __builtin_assume_aligned(p + b * C + code_at, 4 * W), 4 * W);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      __builtin_memcpy(ks[i][b], __builtin_assume_aligned(p + 2 * NB * C + b * 8 + scale_at, 8), 8);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      __builtin_memcpy(v[i][b], __builtin_assume_aligned(p + (NB + b) * C + code_at, 4 * W), 4 * W);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      __builtin_memcpy(vs[i][b], __builtin_assume_aligned(p + 2 * NB * C + NB * 32 + b * 8 + scale_at, 8), 8);
  }
  // operand of K's block b: the lane's token, 8 dimensions
  __device__ __forceinline__ u32x4 k_codes(int i, int b) const {
    if constexpr (Q4) {
      const uint32_t lo = k[i][b][0] & 0x0F0F0F0Fu, hi = k[i][b][0] >> 4 & 0x0F0F0F0Fu;
      return u32x4{codes16<8>(lo, 0x04010400u), codes16<8>(lo, 0x04030402u), codes16<8>(hi, 0x04010400u),
                   codes16<8>(hi, 0x04030402u)};
    } else {
      return u32x4{codes16<128>(k[i][b][0], 0x04010400u), codes16<128>(k[i][b][0], 0x04030402u),
                   codes16<128>(k[i][b][1], 0x04010400u), codes16<128>(k[i][b][1], 0x04030402u)};
    }
  }
  // operand of V's block b, dimensions 16 m .. 16 m + 15: the lane's dimension, 4 + 4 tokens
  __device__ __forceinline__ u32x4 v_codes(int b, int m) const {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (Q4) w[i] = v[i][b][0] >> (4 * m) & 0x0F0F0F0Fu;
      else w[i] = v[i][b][m];
    }
    constexpr int BIAS = Q4 ? 8 : 128;
    return u32x4{codes16<BIAS>(w[0], 0x04010400u), codes16<BIAS>(w[0], 0x04030402u), codes16<BIAS>(w[1], 0x04010400u),
                 codes16<BIAS>(w[1], 0x04030402u)};
  }
};

__device__ __forceinline__ float half_of(const uint32_t (&w)[2], int r) {
  return f16_bits_to_f32(w[r >> 1] >> (16 * (r & 1)) & 0xFFFFu);
}

template <bool Q4, int E, int NB, int TILES, bool PREFIX>
struct Attend {
  static constexpr int QP = E == 0 ? 2 : 1;  // f16 parts of q
  static constexpr int PP = E == 2 ? 1 : 2;  // of a probability times scale
  typedef Step<Q4, E, NB> St;

  u32x4 q[TILES][NB][QP];
  f32x4 o[TILES][NB][2];
  float factor[TILES], ref[TILES], sum[TILES];
  int lo[TILES], hi[TILES];
  int all_lo, all_hi;  // every row of the workgroup sees all_lo .. all_hi - 1

  __device__ __forceinline__ void load_q(const KvAttnArgs& a, int tile, const Row& row, int head, int lane) {
    float x[NB][8];
    uint32_t top = 0;
    if (row.token >= 0) {
      const int64_t at = row.token * a.q_token + head * a.q_head + 8 * (lane >> 4);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (E == 0) {
          __builtin_memcpy(x[b], static_cast<const float*>(a.q) + at + 32 * b, 32);
        } else {
          const u32x4 w = load8(static_cast<const uint16_t*>(a.q) + at + 32 * b);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t bits = w[i];
            x[b][2 * i] = unpack16<E == 1>(bits & 0xFFFFu);
            x[b][2 * i + 1] = unpack16<E == 1>(bits >> 16);
          }
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[b][i] = 0.0f;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, x[b][i]) & 0x7FFFFFFFu);
    top = max(top, uint32_t(__shfl_xor(int(top), 16)));
    top = max(top, uint32_t(__shfl_xor(int(top), 32)));
    // 2^up brings the largest value to [2^14, 2^15); up to 2^126 for f32 that are next to nothing
    const int up = min(126, 14 - (int(top >> 23) - 127));
    const float scale = __builtin_bit_cast(float, uint32_t(127 + up) << 23);
    factor[tile] = top >= 0x7F800000u ? __builtin_nanf("") : a.scale * __builtin_bit_cast(float, uint32_t(127 - up) << 23);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float lowp[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[b][i] *= scale;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = pack16<true>(x[b][2 * i], x[b][2 * i + 1]);
        q[tile][b][0][i] = w;
        lowp[2 * i] = x[b][2 * i] - unpack16<true>(w & 0xFFFFu);
        lowp[2 * i + 1] = x[b][2 * i + 1] - unpack16<true>(w >> 16);
      }
      if constexpr (QP == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[tile][b][1][i] = pack16<true>(lowp[2 * i], lowp[2 * i + 1]);
      }
    }
    lo[tile] = row.token >= 0 ? row.lo : 0;
    hi[tile] = row.token >= 0 ? row.hi : 0x7FFFFFFF;
    ref[tile] = -kInf;
    sum[tile] = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < 2; ++m) o[tile][b][m] = f32x4{0, 0, 0, 0};
  }

  // 32 tokens from position `at`; MASK: some row may not see all of them
  template <bool MASK>
  __device__ __forceinline__ void step(const St& t, int at, int lane) {
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
        const u32x4 k = t.k_codes(i, b);
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          f32x4 d = mfma16<true>(k, q[j][b][0], f32x4{0, 0, 0, 0});
          if constexpr (QP == 2) d = mfma16<true>(k, q[j][b][1], d);
#pragma unroll
          for (int r = 0; r < 4; ++r) s[j][i][r] = fmaf(d[r], half_of(t.ks[i][b], r), s[j][i][r]);
        }
      }
    uint32_t top_scale = 0;
    if constexpr (!MASK) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) top_scale = max_u16(top_scale, max_u16(t.vs[i][b][0], t.vs[i][b][1]));
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
            seen[j][i][r] = t.there[i] && p >= lo[j] && p < hi[j];
            s[j][i][r] = seen[j][i][r] ? s[j][i][r] : -kInf;
#pragma unroll
            for (int b = 0; b < NB; ++b)
              top_v = max(top_v, seen[j][i][r] ? t.vs[i][b][r >> 1] >> (16 * (r & 1)) & 0xFFFFu : 0u);
          }
        }
      if constexpr (!MASK) top_v = max(top_v & 0xFFFFu, top_v >> 16);
      float most = s[j][0][0];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) most = fmaxf(most, s[j][i][r]);
      most += float(int(top_v >> 10 & 31u) - 14);  // V's scales lie below 2^(exponent - 14)
      if (__builtin_expect(__any(most > ref[j] + 15.0f), 0)) {
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
      const u32x4 v0 = t.v_codes(b, 0), v1 = t.v_codes(b, 1);
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        float pv[8];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float sv = half_of(t.vs[i][b], r);
            if constexpr (MASK) sv = seen[j][i][r] ? sv : 0.0f;
            pv[4 * i + r] = s[j][i][r] * sv;
          }
        u32x4 p, pl;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = pack16<true>(pv[2 * i], pv[2 * i + 1]);
          if constexpr (PP == 2)
            pl[i] = pack16<true>(pv[2 * i] - unpack16<true>(p[i] & 0xFFFFu), pv[2 * i + 1] - unpack16<true>(p[i] >> 16));
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
};

// Row r of the tile: its token and the positions it sees in [from, to).
template <bool PREFIX>
__device__ __forceinline__ Row row_of(const KvAttnArgs& a, uint32_t r, uint32_t rows, int first_row, int64_t first_pos,
                                      int from, int64_t cap) {
  Row w{-1, 0, 0};
  if (r >= rows) return w;
  const int i = int(r / uint32_t(a.group));
  int64_t pos;
  w.token = first_row + i;
  if constexpr (PREFIX) {  // its sequence by bisection
    int x = 0, n = a.kv.B;
    while (n > 1) {
      const int h = n >> 1;
      if (kv_row_start(a.kv, x + h) <= w.token) x += h, n -= h;
      else n = h;
    }
    const int end = kv_row_start(a.kv, x + 1);
    if (w.token < kv_row_start(a.kv, x) || w.token >= end) return Row{-1, 0, 0};
    pos = int64_t(a.kv.kv_len[x]) - end + w.token;
  } else {
    pos = first_pos + i;
  }
  const int64_t lo = a.window ? max(int64_t(0), pos - a.window + 1) : 0;
  w.lo = int(min(max(lo, int64_t(from)), cap));
  w.hi = int(max(int64_t(0), min(pos + 1, cap)));
  return w;
}

// grid: (k / v heads * splits * sequences (1 for the prefix), row blocks)
template <bool Q4, int E, int NB, int TILES, bool PREFIX>
__global__ __launch_bounds__(256, 2) void kv_attention_kernel(const KvAttnArgs a, int splits, int first_slot) {
  typedef Attend<Q4, E, NB, TILES, PREFIX> At;
  typedef typename At::St St;
  __shared__ f32x4 meet[3][NB * 2][64];
  __shared__ float2 meet_stats[3][64];
  constexpr int kRows = 16 * TILES;
  const KvArgs& kv = a.kv;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = blockIdx.x / kv.heads, head = blockIdx.x - item * kv.heads;
  const int b = PREFIX ? 0 : item / splits, split = item - b * splits;
  const int r0 = PREFIX ? 0 : kv_row_start(kv, b);
  const int r1 = PREFIX ? kv_row_start(kv, kv.B) : max(r0, kv_row_start(kv, b + 1));
  const uint32_t rows = uint32_t(r1 - r0) * uint32_t(a.group);  // below 2^31
  const int64_t cap64 = int64_t(kv.columns) * kv.sets * 16;
  const int64_t cap = PREFIX ? min(cap64, int64_t(a.prefix)) : cap64;
  const int64_t first_pos = PREFIX ? 0 : int64_t(kv.kv_len[b]) - (r1 - r0);
  const int32_t* table = kv.table + (PREFIX ? 0 : b * kv.stride);

  for (uint32_t base = blockIdx.y * kRows; base < rows; base += gridDim.y * kRows) {
    At w;
    int most_lo = 0, least_hi = 0x7FFFFFFF, least_lo = 0x7FFFFFFF, most_hi = 0;
    Row row[TILES];
    int row_head[TILES];
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const uint32_t r = base + 16 * j + (lane & 15);
      row[j] = row_of<PREFIX>(a, r, rows, r0, first_pos, PREFIX ? 0 : a.prefix, cap);
      if (row[j].token >= 0) {
        most_lo = max(most_lo, row[j].lo);
        least_hi = min(least_hi, row[j].hi);
        if (row[j].lo < row[j].hi) {
          least_lo = min(least_lo, row[j].lo);
          most_hi = max(most_hi, row[j].hi);
        }
      }
      row_head[j] = head * a.group + int(r % uint32_t(a.group));
      w.load_q(a, j, row[j], row_head[j], lane);
    }
    w.all_lo = wave_max(most_lo);
    w.all_hi = -wave_max(-least_hi);
    least_lo = -wave_max(-least_lo);
    most_hi = wave_max(most_hi);
    // the sets of 16 tokens that any row sees, and this split's share of them: whole steps of all waves
    const int s0 = least_lo < most_hi ? least_lo >> 4 : 0, s1 = least_lo < most_hi ? (most_hi + 15) >> 4 : 0;
    const int share = ((s1 - s0 + splits - 1) / splits + 7) & ~7;
    const int u0 = s0 + split * share, u1 = min(s1, u0 + share);
    const int steps = u1 > u0 + 2 * wave ? (u1 - u0 - 2 * wave + 7) >> 3 : 0;  // of this wave: sets u0 + 2 wave + 8 n

    // pages of the wave's next 32 steps: lane 2 n + i holds the page of set i of step n
    int pages = -1, places = 0;
    auto look_up = [&](int n0) {
      const int u = u0 + 2 * wave + 8 * (n0 + (lane >> 1)) + (lane & 1);
      int set, page = -1;
      const int p = kv_page_of(kv, uint32_t(min(u, s1 - 1)), set);
      if (u < u1) {
        page = table[p];
        if (page < 0 || page >= kv.pages) page = -1;
      }
      pages = page;
      places = set;
    };
    auto fetch = [&](St& t, int n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int l = 2 * (n & 31) + i;
        t.load(kv, head, i, __builtin_amdgcn_readlane(pages, l), __builtin_amdgcn_readlane(places, l), lane);
      }
    };
    auto work = [&](const St& t, int n) {
      const int at = (u0 + 2 * wave + 8 * n) * 16;
      if (t.there[0] && t.there[1] && at >= w.all_lo && at + 32 <= w.all_hi) w.template step<false>(t, at, lane);
      else w.template step<true>(t, at, lane);
    };
    if (steps > 0) {
      look_up(0);
      St one, two;
      fetch(one, 0);
      for (int n = 0; n < steps; n += 2) {
        if (n + 1 < steps) fetch(two, n + 1);
        work(one, n);
        if (n + 2 < steps) {
          if (((n + 2) & 31) == 0) look_up(n + 2);
          fetch(one, n + 2);
        }
        if (n + 1 < steps) work(two, n + 1);
      }
    }

    // the four waves meet: wave j % 4 joins tile j
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      w.sum[j] = column_sum(w.sum[j]);
      const int owner = j & 3, slot = wave < owner ? wave : wave - 1;
      if (wave != owner) {
#pragma unroll
        for (int i = 0; i < NB * 2; ++i) meet[slot][i][lane] = w.o[j][i >> 1][i & 1];
        meet_stats[slot][lane] = make_float2(w.ref[j], w.sum[j]);
      }
      __syncthreads();
      if (wave == owner) {
        float ref = w.ref[j];
#pragma unroll
        for (int k = 0; k < 3; ++k) ref = fmaxf(ref, meet_stats[k][lane].x);
        const float from = ref == -kInf ? 0.0f : ref;
        const float f = __builtin_amdgcn_exp2f(w.ref[j] - from);
        float sum = w.sum[j] * f;
#pragma unroll
        for (int i = 0; i < NB * 2; ++i) w.o[j][i >> 1][i & 1] *= f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const float2 st = meet_stats[k][lane];
          const float g = __builtin_amdgcn_exp2f(st.x - from);
          sum = fmaf(st.y, g, sum);
#pragma unroll
          for (int i = 0; i < NB * 2; ++i) {
            const f32x4 v = meet[k][i][lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) w.o[j][i >> 1][i & 1][r] = fmaf(v[r], g, w.o[j][i >> 1][i & 1][r]);
          }
        }
        if (row[j].token >= 0) {
          const int h = row_head[j];
          const int64_t at = row[j].token * int64_t(a.q_heads) + h;
          if (a.slots) {
            const int64_t part = at * a.slots + first_slot + split;
            if (lane < 16) a.stats[part] = make_float2(ref, sum);
            if (sum != 0.0f) {  // nothing seen: the join does not look at it
#pragma unroll
              for (int i = 0; i < NB * 2; ++i)
                *reinterpret_cast<f32x4*>(a.sums + part * (32 * NB) + 16 * i + 4 * (lane >> 4)) = w.o[j][i >> 1][i & 1];
            }
          } else {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (a.lse && lane < 16)
              a.lse[at] = sum == 0.0f ? -kInf : 0.69314718f * (ref + __builtin_amdgcn_logf(sum));
            const int64_t to = row[j].token * a.out_token + h * a.out_head + 4 * (lane >> 4);
#pragma unroll
            for (int i = 0; i < NB * 2; ++i) {
              f32x4 v = w.o[j][i >> 1][i & 1] * inv;
              if (sum == 0.0f) v = f32x4{0, 0, 0, 0};
              if constexpr (E == 0) {
                __builtin_memcpy(static_cast<float*>(a.out) + to + 16 * i, &v, 16);
              } else {
                const u32x2 x = {pack16<E == 1>(v[0], v[1]), pack16<E == 1>(v[2], v[3])};
                __builtin_memcpy(static_cast<uint16_t*>(a.out) + to + 16 * i, &x, 8);
              }
            }
          }
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace

// One head size's launch; tiles 1 or 2.
template <bool Q4, int E, int NB>
hipError_t kv_attention_go(const KvAttnArgs& a, const KvAttentionPlan& p, hipStream_t s) {
  const unsigned heads = unsigned(a.kv.heads);
  if (a.prefix) {
    const dim3 grid(heads * unsigned(p.prefix_splits), unsigned(p.prefix_row_blocks), 1);
    if (p.prefix_tiles == 1) hipLaunchKernelGGL((kv_attention_kernel<Q4, E, NB, 1, true>), grid, dim3(256), 0, s, a, p.prefix_splits, 0);
    else hipLaunchKernelGGL((kv_attention_kernel<Q4, E, NB, 2, true>), grid, dim3(256), 0, s, a, p.prefix_splits, 0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int first = a.prefix ? p.prefix_splits : 0;
  const dim3 grid(heads * unsigned(p.splits) * unsigned(a.kv.B), unsigned(p.row_blocks), 1);
  if (p.tiles == 1) hipLaunchKernelGGL((kv_attention_kernel<Q4, E, NB, 1, false>), grid, dim3(256), 0, s, a, p.splits, first);
  else hipLaunchKernelGGL((kv_attention_kernel<Q4, E, NB, 2, false>), grid, dim3(256), 0, s, a, p.splits, first);
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
