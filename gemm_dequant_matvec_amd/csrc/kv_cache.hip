// Writing keys and values into the quantised cache, and reading them back.
//
//   d = f16(max |x| / s), q = rint(x * (1 / d))   (blocks of 32 values of a head)
//
// Bound by memory.  Sixteen lanes take a block of the 16 tokens of a set, four of
// them a group of four tokens: each holds 8 dimensions of the four tokens, the
// block's maximum of a token is a four-lane maximum, and what a lane writes (or
// reads) of the cache is then one run of 32 bytes (Q4_0: 16): for K the dimensions
// 8 j .. 8 j + 7 of the four tokens, for V the dimensions 4 j .. 4 j + 3 and
// 16 + 4 j .. of the four.  The sixteen lanes' runs are the block's codes without a
// gap.  A group of which the call has only some tokens (a single new token, the ends
// of a prompt) is written in bytes, and only theirs.  The division for a block's scale
// and the one for its inverse are made by one lane for each of the four tokens.
//
// A workgroup takes a set of a sequence, its 16 x 16 lanes the set's (head, k or v,
// block) items, so that whole lines of the cache come from one workgroup.  Sets are
// counted so that the workgroup of a set follows from q_start alone: sequence b
// starts at set q_start[b] / 16 + 2 b, which leaves room for the ends of both sides,
// and T / 16 + 2 B sets are launched.
//
// Write and read back of 8 ragged prompts (11000 tokens, 8 heads of 128, bf16, Q4_0): 97 us,
// 4.3 TB/s of what the two have to move; read of 24 ragged sequences (Q8_0): 231 us, 4.9 TB/s.
// (A group of four tokens per wave, so that a line comes from several workgroups: 143 and 291.)
#include <algorithm>

#include "cache_internal.h"
#include "rope.h"

namespace qmv {
namespace {

constexpr int kThreads = 256;

struct KvHeads {  // k or v of the new tokens, or where they are read to; NULL: not wanted
  const void* p;
  int64_t token, head;
};

// The four tokens of a group: which are the call's, and where they lie.
struct Group {
  int head_at;      // bytes from the page's head to the group's set; -1: the group is not there
  int64_t page_at;  // bytes from the cache to the page
  int t4;           // group of the set
  int row, from, to;  // row of token 0, tokens from .. to - 1 are the call's
};

// The group t4 of set v.
__device__ __forceinline__ bool group_of(const KvArgs& a, int64_t v, int t4, Group& g) {
  const int b = kv_search(a.B, v, [&](int i) { return int64_t(kv_row_start(a, i) >> 4) + 2 * int64_t(i); });
  const int r0 = kv_row_start(a, b), r1 = max(r0, kv_row_start(a, b + 1)), n = r1 - r0;
  const int64_t first = int64_t(a.kv_len[b]) - n;  // position of row r0
  // sets are counted from the first position's, rounded down (also below 0)
  const int64_t s = ((first >> 4) + (v - ((r0 >> 4) + 2 * int64_t(b)))) * 16, p = s + 4 * t4;  // position of token 0
  g.from = int(min(int64_t(4), max(int64_t(0), first - p)));
  g.to = int(max(int64_t(0), min(int64_t(4), first + n - p)));
  g.row = int(r0 + (p - first));
  g.t4 = t4;
  g.head_at = -1;
  if (s >= first + n) return false;
  if (s >= 0 && s < int64_t(a.columns) * a.sets * 16) {  // sets do not straddle position 0
    int set;
    const int page = kv_page_of(a, uint32_t(s >> 4), set);
    const int id = a.table[b * a.stride + page];
    if (id >= 0 && id < a.pages) {
      g.head_at = set * a.set_bytes;
      g.page_at = id * a.page_bytes;
    }
  }
  return true;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, true)));
}

// Lane T of the quad's.
template <int T>
__device__ __forceinline__ uint32_t of_lane(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), T * 0x55, 0xF, 0xF, true));
}
// The lowest bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
}

// Dimension of value i (0 .. 7) of lane j of a quad.
template <bool V>
__device__ __forceinline__ int dim_of(int j, int i) {
  return V ? 4 * j + (i & 3) + 16 * (i >> 2) : 8 * j + i;
}
template <int E, bool V>
__device__ __forceinline__ void load8_of(const typename Elem<E>::T* p, int j, float (&x)[8]) {
  if constexpr (E == 0) {
    float lo[4], hi[4];
    Elem<0>::load(p + dim_of<V>(j, 0), 4, lo);
    Elem<0>::load(p + dim_of<V>(j, 4), 4, hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = lo[i], x[4 + i] = hi[i];
  } else {
    uint32_t w[4];
    __builtin_memcpy(w, p + dim_of<V>(j, 0), 8);
    __builtin_memcpy(w + 2, p + dim_of<V>(j, 4), 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = unpack16<E == 1>(w[i] & 0xFFFFu);
      x[2 * i + 1] = unpack16<E == 1>(w[i] >> 16);
    }
  }
}
template <int E, bool V>
__device__ __forceinline__ void store8_of(typename Elem<E>::T* p, int j, const float (&x)[8]) {
  if constexpr (E == 0) {
    __builtin_memcpy(p + dim_of<V>(j, 0), x, 16);
    __builtin_memcpy(p + dim_of<V>(j, 4), x + 4, 16);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack16<E == 1>(x[2 * i], x[2 * i + 1]);
    __builtin_memcpy(p + dim_of<V>(j, 0), w, 8);
    __builtin_memcpy(p + dim_of<V>(j, 4), w + 2, 8);
  }
}

// One item: block `blk` of a head of K or V, its four tokens.  rec: the set's record.
template <int E, bool Q4, bool V>
__device__ __forceinline__ void write_item(const KvArgs& a, const Group& g, uint8_t* rec, const KvHeads& src, int head,
                                           int blk, int j) {
  constexpr int C = Q4 ? 256 : 512, W = Q4 ? 4 : 8;  // words that a lane writes
  constexpr float kTop = Q4 ? 7.0f : 127.0f, kLow = Q4 ? -8.0f : -127.0f, kSpan = Q4 ? 7.5f : 127.0f;
  uint32_t code[4][8];  // in the lowest byte: four tokens, 8 values each
  uint32_t scale[4], top[4];
  float x[4][8];
  typedef typename Elem<E>::T T;
  const T* p = static_cast<const T*>(src.p) + head * src.head + 32 * blk;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (t >= g.from && t < g.to) {
      load8_of<E, V>(p + int64_t(g.row + t) * src.token, j, x[t]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[t][i] = 0.0f;
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    top[t] = 0;  // as bits: NaN > infinity > numbers
#pragma unroll
    for (int i = 0; i < 8; ++i) top[t] = max(top[t], __builtin_bit_cast(uint32_t, x[t][i]) & 0x7FFFFFFFu);
    top[t] = dpp_max<0x4E>(dpp_max<0xB1>(top[t]));
  }
  const uint32_t mine = j & 2 ? (j & 1 ? top[3] : top[2]) : (j & 1 ? top[1] : top[0]);
  const bool bad = mine >= 0x7F800000u;
  const _Float16 d = static_cast<_Float16>(fminf(__builtin_bit_cast(float, mine) / kSpan, 65504.0f));
  const float df = static_cast<float>(d);
  const uint32_t inv = __builtin_bit_cast(uint32_t, df > 0.0f && !bad ? 1.0f / df : 0.0f);
  const uint32_t bits = bad ? 0x7E00u : uint32_t(__builtin_bit_cast(uint16_t, d));
  const float by[4] = {__builtin_bit_cast(float, of_lane<0>(inv)), __builtin_bit_cast(float, of_lane<1>(inv)),
                       __builtin_bit_cast(float, of_lane<2>(inv)), __builtin_bit_cast(float, of_lane<3>(inv))};
  scale[0] = of_lane<0>(bits), scale[1] = of_lane<1>(bits), scale[2] = of_lane<2>(bits), scale[3] = of_lane<3>(bits);
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // next to 1.5 2^23 an f32 step is 1: the sum rounds to the even neighbour as rint does, and ends in q + 128 (q + 8)
      const float q = top[t] >= 0x7F800000u ? 0.0f : __builtin_amdgcn_fmed3f(x[t][i] * by[t], kLow, kTop);
      code[t][i] = __builtin_bit_cast(uint32_t, q + (12582912.0f + (Q4 ? 8.0f : 128.0f)));
    }
  const int nb = a.nb;
  uint8_t* dst = rec + (V ? nb * C : 0) + blk * C;
  uint8_t* sc = rec + 2 * nb * C + (V ? nb * 32 : 0) + (g.t4 * nb + blk) * 8;
  const bool full = g.from == 0 && g.to == 4;
  if constexpr (!V) {  // token t: W / 4 words of its 8 codes
    dst += (16 * j + 4 * g.t4) * W;
    uint32_t w[W];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t lo = low_bytes(code[t][0], code[t][1], code[t][2], code[t][3]);
      const uint32_t hi = low_bytes(code[t][4], code[t][5], code[t][6], code[t][7]);
      if constexpr (Q4) w[t] = lo | hi << 4;
      else w[2 * t] = lo, w[2 * t + 1] = hi;
    }
    if (full) {
#pragma unroll
      for (int i = 0; i < W; i += 4) *reinterpret_cast<u32x4*>(dst + 4 * i) = u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t >= g.from && t < g.to) {
          if constexpr (Q4) *reinterpret_cast<uint32_t*>(dst + 4 * t) = w[t];
          else *reinterpret_cast<u32x2*>(dst + 8 * t) = u32x2{w[2 * t], w[2 * t + 1]};
        }
    }
  } else {  // dimension 4 j + i, then (Q8_0) 16 + 4 j + i: a word of four tokens each
    dst += (16 * g.t4 + 4 * j) * W;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = low_bytes(code[0][i], code[1][i], code[2][i], code[3][i]);
      const uint32_t hi = low_bytes(code[0][4 + i], code[1][4 + i], code[2][4 + i], code[3][4 + i]);
      if constexpr (Q4) w[i] = lo | hi << 4;
      else w[2 * i] = lo, w[2 * i + 1] = hi;
    }
    if (full) {
#pragma unroll
      for (int i = 0; i < W; i += 4) *reinterpret_cast<u32x4*>(dst + 4 * i) = u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t >= g.from && t < g.to) {
#pragma unroll
          for (int i = 0; i < W; ++i) dst[4 * i + t] = uint8_t(w[i] >> (8 * t));
        }
    }
  }
  if (j == 0) {
    if (full) {
      *reinterpret_cast<u32x2*>(sc) = u32x2{scale[0] | scale[1] << 16, scale[2] | scale[3] << 16};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t >= g.from && t < g.to) reinterpret_cast<uint16_t*>(sc)[t] = uint16_t(scale[t]);
    }
  }
}

template <int E, bool Q4, bool V>
__device__ __forceinline__ void read_item(const KvArgs& a, const Group& g, const uint8_t* rec, const KvHeads& dst, int head,
                                          int blk, int j) {
  constexpr int C = Q4 ? 256 : 512, W = Q4 ? 4 : 8;
  typedef typename Elem<E>::T T;
  T* p = static_cast<T*>(const_cast<void*>(dst.p)) + head * dst.head + 32 * blk;
  uint32_t w[W];
  uint32_t sw[2] = {0, 0};
  if (rec) {
    const int nb = a.nb;
    const uint8_t* src = rec + (V ? nb * C : 0) + blk * C + (V ? 16 * g.t4 + 4 * j : 16 * j + 4 * g.t4) * W;
    __builtin_memcpy(w, __builtin_assume_aligned(src, 16), 4 * W);
    __builtin_memcpy(sw, __builtin_assume_aligned(rec + 2 * nb * C + (V ? nb * 32 : 0) + (g.t4 * nb + blk) * 8, 8), 8);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (t < g.from || t >= g.to) continue;
    const float d = f16_bits_to_f32(sw[t >> 1] >> (16 * (t & 1)) & 0xFFFFu);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t q;
      if constexpr (!V && Q4) q = w[t] >> (8 * (i & 3) + 4 * (i >> 2)) & 15u;
      else if constexpr (!V) q = w[2 * t + (i >> 2)] >> (8 * (i & 3)) & 255u;
      else if constexpr (Q4) q = w[i & 3] >> (8 * t + 4 * (i >> 2)) & 15u;
      else q = w[2 * (i & 3) + (i >> 2)] >> (8 * t) & 255u;
      x[i] = rec ? float(int(q) - (Q4 ? 8 : 128)) * d : 0.0f;
    }
    store8_of<E, V>(p + int64_t(g.row + t) * dst.token, j, x);
  }
}

template <int E, bool Q4, bool WRITE>
__global__ __launch_bounds__(kThreads) void kv_cache_kernel(const KvArgs a, const KvHeads k, const KvHeads v) {
  const int slot = threadIdx.x >> 4, t4 = threadIdx.x >> 2 & 3, j = threadIdx.x & 3;
  const int64_t sets = (int64_t(a.T) >> 4) + 2 * int64_t(a.B);
  for (int64_t n = blockIdx.x; n < sets; n += gridDim.x) {
    Group g;
    if (!group_of(a, n, t4, g)) continue;
    const bool there = g.head_at >= 0;
    if (WRITE && !there) continue;
    if (g.from >= g.to) continue;
    const int items = a.heads * 2 * a.nb;
    for (int it = slot; it < items; it += 16) {
      const int hv = it / a.nb, blk = it - hv * a.nb, h = hv >> 1;
      uint8_t* rec = there ? a.data + g.page_at + int64_t(h) * a.head_bytes + g.head_at : nullptr;
      if constexpr (WRITE) {
        if (hv & 1) write_item<E, Q4, true>(a, g, rec, v, h, blk, j);
        else write_item<E, Q4, false>(a, g, rec, k, h, blk, j);
      } else {
        if (hv & 1) {
          if (v.p) read_item<E, Q4, true>(a, g, rec, v, h, blk, j);
        } else {
          if (k.p) read_item<E, Q4, false>(a, g, rec, k, h, blk, j);
        }
      }
    }
  }
}

template <bool WRITE>
hipError_t launch(const qmv_kv_cache& c, const qmv_kv_batch& b, const KvHeads& k, const KvHeads& v, int dtype, hipStream_t s) {
  const KvArgs a = kv_args(c, b);
  const dim3 grid(unsigned(std::min<int64_t>((b.T >> 4) + 2 * b.B, 1 << 20)));
  auto go = [&](auto e) {
    constexpr int E = decltype(e)::value;
    if (c.fmt == QMV_Q4_0) hipLaunchKernelGGL((kv_cache_kernel<E, true, WRITE>), grid, dim3(kThreads), 0, s, a, k, v);
    else hipLaunchKernelGGL((kv_cache_kernel<E, false, WRITE>), grid, dim3(kThreads), 0, s, a, k, v);
  };
  if (dtype == QMV_F32) go(std::integral_constant<int, 0>{});
  else if (dtype == QMV_F16) go(std::integral_constant<int, 1>{});
  else go(std::integral_constant<int, 2>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_write(const qmv_kv_cache& c, const qmv_kv_batch& b, const void* k, int64_t k_token, int64_t k_head,
                           const void* v, int64_t v_token, int64_t v_head, int dtype, hipStream_t s) {
  return launch<true>(c, b, KvHeads{k, k_token, k_head}, KvHeads{v, v_token, v_head}, dtype, s);
}

hipError_t launch_kv_read(const qmv_kv_cache& c, const qmv_kv_batch& b, void* k, int64_t k_token, int64_t k_head, void* v,
                          int64_t v_token, int64_t v_head, int dtype, hipStream_t s) {
  return launch<false>(c, b, KvHeads{k, k_token, k_head}, KvHeads{v, v_token, v_head}, dtype, s);
}

}  // namespace qmv
