// Shared by the many-token products (glu_fwd*.hip, glu_bwd*.hip): the 16-bit
// types, the matrix-core fragments, the LDS tile and the decoding of packed
// weights to the 16-bit operand type.
//
// Every format's weight is w = a * t + b with a code byte t in 0..255 and f32
// (a, b) per 32-weight unit (per 16 weights in Q6K); one fma gives the value of
// the format's definition: a * t is exact or the only rounding is the one the
// definition has too (W4A16: s q - s z with s z exact; Q4K, Q5K: the one
// subtraction; per-row int8: s t - 128 s = s q rounded once).  It is then
// rounded once, to nearest even, to the operand type.
#pragma once

#include "layer_internal.h"

namespace qmv {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two f32 to two 16-bit values, round to nearest even, first in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  const f32x2 v = {a, b};
  if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <bool F16>
__device__ __forceinline__ float unpack16(uint32_t bits) {  // low 16 bits
  if constexpr (F16) return f16_bits_to_f32(bits & 0xFFFFu);
  else return bf16_bits_to_f32(bits);
}

template <bool F16>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {  // 32x32, 16 deep
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {  // 16x16, 32 deep
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Workgroup barrier for LDS traffic only (global loads stay in flight).
__device__ __forceinline__ void lds_barrier16() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 16-byte load of eight 16-bit values at any 2-byte aligned address.
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// The first n (1..7) of eight 16-bit values at p, zeros behind them; nothing
// past p[n - 1] is read (the last value again instead: eight loads that are
// under way together, where a branch per value waits for each).
__device__ __forceinline__ u32x4 load_part(const uint16_t* p, int n) {
  uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t v = p[min(e, n - 1)];
    o[e >> 1] |= e < n ? v << (16 * (e & 1)) : 0u;
  }
  return u32x4{o[0], o[1], o[2], o[3]};
}

// ------------------------------------------------------------------ LDS tile
// Rows of 64 16-bit values (128 bytes, eight 16-byte pieces).  16 lanes reach
// all 64 banks at once if their pieces differ in address bits 4..7.  Piece c of
// row r sits at c ^ (r / 2 % 8) of its row: by the banks, no two of 16
// consecutive rows meet in one piece, and a fragment 32 rows on is a constant offset
// away.
__device__ __forceinline__ int tile_at(int r, int c) {  // in 16-byte pieces
  return r * 8 + (c ^ ((r >> 1) & 7));
}
// The same for rows of 32 values (64 bytes, four pieces).  Counted conflict cycles
// per LDS instruction of the forward kernel, W4A16: 0.28 with the 64 x 256 tile, 1.1
// with 128 x 256, in the loop (K = 4096 against 2048: 24.2 M against 12.6 M; the
// epilogue is 1.1 M of them): 16 cycles per wave and stage against 2.  The larger
// tile's decoders differ: two threads, not four, share a row and write pieces two
// apart, so that eight neighbouring lanes meet in pairs; 7 cycles per such write
// would be the whole.
__device__ __forceinline__ int tile32_at(int r, int c) {
  return r * 4 + (c ^ ((r >> 2) & 3));
}

// -------------------------------------------------------- workgroups to tiles
// Consecutive workgroups go to the 8 XCDs in turn, each with an L2 of its own.
// Here an XCD takes a contiguous eighth of the tiles, and tiles count through
// bands of kBand token tiles, so the 32 tiles an XCD works on at a time share 4
// token and 8 weight tiles.
struct TileId {
  int x, y;
};
constexpr int kBand = 4;
__device__ __forceinline__ TileId tile_of_block(int nx, int bx, int ny, int by) {
  const int X = (nx + bx - 1) / bx, Y = (ny + by - 1) / by, all = X * Y;
  const int b = blockIdx.x, xcd = b & 7, per = all >> 3, more = all & 7;
  const int t = xcd * per + min(xcd, more) + (b >> 3);  // XCD i takes per tiles, the first `more` one extra
  const int band = t / (kBand * X), in = t - band * kBand * X;
  const int high = min(kBand, Y - band * kBand);
  return TileId{in / high, band * kBand + in % high};
}

// ------------------------------------------------------------ packed weights

struct Mat {  // one packed matrix on the device
  const uint8_t* p[4];
};

inline Mat mat_of(const uint8_t* W, const Planes& p) {
  Mat m;
  for (int i = 0; i < 4; ++i) m.p[i] = W + p.off[i];
  return m;
}

// Bytes of one row of plane i.
template <int FMT>
__device__ __forceinline__ uint32_t row_bytes(int i, int K) {
  if constexpr (FMT == QMV_Q8_0) return i ? K >> 4 : K;
  else if constexpr (FMT == QMV_Q6K) return i == 0 ? K >> 1 : i == 1 ? K >> 2 : i == 2 ? K >> 4 : K >> 7;
  else if constexpr (FMT == QMV_Q5_0 || FMT == QMV_Q5K) return i == 0 ? K >> 1 : i == 1 ? K >> 3 : K >> 4;
  else if constexpr (FMT == QMV_DENSE_BF16) return 2 * K;
  else if constexpr (FMT == QMV_I8_ROW) return i ? 4 : K;
  else return i ? K >> 4 : K >> 1;  // W4A16_G64, Q4K, Q4_0
}

template <int FMT>
constexpr int kPlanes = FMT == QMV_DENSE_BF16 ? 1 : FMT == QMV_Q6K ? 4 : FMT == QMV_Q5_0 || FMT == QMV_Q5K ? 3 : 2;

// The matrix from row n on.  Loads below take a row relative to it, so that
// with a uniform n every address is a scalar base and a 32-bit lane offset.
template <int FMT>
__device__ __forceinline__ Mat from_row(const Mat& w, int64_t n, int K) {
  Mat m;
#pragma unroll
  for (int i = 0; i < kPlanes<FMT>; ++i) m.p[i] = w.p[i] + n * row_bytes<FMT>(i, K);
  return m;
}

// Keeps a uniform address in scalar registers: without it the compiler adds the
// lane offset first and carries a 64-bit address per lane and load through the
// loop (and spills them).
#define QMV_GLOBAL __attribute__((address_space(1)))
__device__ __forceinline__ const QMV_GLOBAL uint8_t* scalar_base(const uint8_t* p) {
  const QMV_GLOBAL uint8_t* g = (const QMV_GLOBAL uint8_t*)p;
  asm volatile("" : "+s"(g));
  return g;
}

// Keeps the widening of a lane offset next to its use, where it folds into the
// address (hoisted out of the loop it becomes a 64-bit value per lane).
__device__ __forceinline__ uint32_t lane_offset(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// How the addresses of a load differ between the lanes of a wave: only in the
// row; in the row and in u, which then joins the 32-bit offset instead of the
// scalar base; or in the matrix too.
enum By { kByRow, kByUnit, kByMatrix };

// A T at byte `row` (a lane's) + `u` of a plane.
template <class T, By BY = kByUnit>
__device__ __forceinline__ T load_at(const uint8_t* plane, uint32_t row, int64_t u = 0) {
  if constexpr (BY == kByMatrix) return *reinterpret_cast<const T*>(plane + (row + uint32_t(u)));
  else if constexpr (BY == kByUnit) return *(const QMV_GLOBAL T*)(scalar_base(plane) + lane_offset(row + uint32_t(u)));
  else return *(const QMV_GLOBAL T*)(scalar_base(plane + u) + lane_offset(row));
}

struct Affine {  // w = a t + b; a1, b1 for the second 16 weights (Q6K), else as a0, b0
  float a0, b0, a1, b1;
};

constexpr bool is_byte(int fmt) { return fmt == QMV_Q8_0 || fmt == QMV_I8_ROW; }
constexpr bool is_fifth(int fmt) { return fmt == QMV_Q5_0 || fmt == QMV_Q5K; }
constexpr bool is_super(int fmt) { return fmt == QMV_Q4K || fmt == QMV_Q5K; }

// What the scales of one unit are loaded as.
template <int FMT>
struct MetaRaw {
  u32x4 v;  // super-block record, or v[0], v[1]
};

// Byte offsets of a row in each plane.
template <int FMT>
struct RowAt {
  uint32_t o[kPlanes<FMT>];
};

template <int FMT>
__device__ __forceinline__ RowAt<FMT> row_at(uint32_t r, int K) {
  RowAt<FMT> x;
#pragma unroll
  for (int i = 0; i < kPlanes<FMT>; ++i) x.o[i] = r * row_bytes<FMT>(i, K);
  return x;
}

// The scales of unit u of a row.
template <int FMT, By BY>
__device__ __forceinline__ MetaRaw<FMT> load_meta(const Mat& w, const RowAt<FMT>& r, int u) {
  MetaRaw<FMT> m;
  constexpr int P = kPlanes<FMT> - 1;  // the plane of the scales (Q6K: of d)
  const uint32_t at = r.o[P];
  if constexpr (FMT == QMV_Q8_0 || FMT == QMV_Q4_0 || FMT == QMV_Q5_0) {
    m.v[0] = load_at<uint16_t, BY>(w.p[P], at, 2 * u);
  } else if constexpr (FMT == QMV_W4A16_G64) {
    m.v[0] = load_at<uint32_t, BY>(w.p[P], at, 4 * (u >> 1));
  } else if constexpr (is_super(FMT)) {
    m.v = load_at<u32x4, BY>(w.p[P], at, 16 * (u >> 3));
  } else if constexpr (FMT == QMV_Q6K) {
    m.v[0] = load_at<uint16_t, BY>(w.p[2], r.o[2], 2 * u);
    m.v[1] = load_at<uint16_t, BY>(w.p[3], at, 2 * (u >> 3));
  } else if constexpr (FMT == QMV_I8_ROW) {
    m.v[0] = load_at<uint32_t, BY>(w.p[1], at);
  }
  return m;
}

template <int FMT>
__device__ __forceinline__ Affine affine_of(const MetaRaw<FMT>& m, int u) {
  Affine f{0.f, 0.f, 0.f, 0.f};
  if constexpr (FMT == QMV_Q8_0) {
    f.a0 = f16_bits_to_f32(m.v[0]);
    f.b0 = -128.0f * f.a0;
  } else if constexpr (FMT == QMV_Q4_0 || FMT == QMV_Q5_0) {
    f.a0 = f16_bits_to_f32(m.v[0]);
    f.b0 = (FMT == QMV_Q4_0 ? -8.0f : -16.0f) * f.a0;
  } else if constexpr (FMT == QMV_W4A16_G64) {
    f.a0 = f16_bits_to_f32(m.v[0] & 0xFFFFu);
    f.b0 = -(f.a0 * f16_bits_to_f32(m.v[0] >> 16));
  } else if constexpr (is_super(FMT)) {
    const uint32_t r1 = m.v[1], r2 = m.v[2], r3 = m.v[3];
    const int sh = 6 * (u & 7);
    const uint64_t lo = uint64_t(r1) | (uint64_t(r2) << 32);        // bits 0..63 of the 96
    const uint64_t hi = uint64_t(r2 >> 16) | (uint64_t(r3) << 16);  // bits 48..95
    f.a0 = f16_bits_to_f32(m.v[0] & 0xFFFFu) * static_cast<float>(uint32_t(lo >> sh) & 63u);
    f.b0 = -(f16_bits_to_f32(m.v[0] >> 16) * static_cast<float>(uint32_t(hi >> sh) & 63u));
  } else if constexpr (FMT == QMV_Q6K) {
    const float d = f16_bits_to_f32(m.v[1]);
    f.a0 = d * static_cast<float>(static_cast<int8_t>(m.v[0] & 0xFFu));
    f.a1 = d * static_cast<float>(static_cast<int8_t>((m.v[0] >> 8) & 0xFFu));
    f.b0 = -32.0f * f.a0;
    f.b1 = -32.0f * f.a1;
  } else if constexpr (FMT == QMV_I8_ROW) {
    const uint32_t s = m.v[0];
    f.a0 = __builtin_bit_cast(float, s);
    f.b0 = -128.0f * f.a0;
  }
  return f;
}

// The codes of eight weights as loaded: q0 (and q1 for 8-bit codes) and the
// word that holds their higher bits.
struct Word8 {
  uint32_t q0, q1, qh;
};

// Eight weights a t + b of word i (0..3) of a unit, in f32.
template <int FMT>
__device__ __forceinline__ void decode8(const Word8& c, float a, float b, int i, float (&w)[8]) {
  if constexpr (is_byte(FMT)) {
    const uint32_t lo = c.q0 ^ 0x80808080u, hi = c.q1 ^ 0x80808080u;  // q + 128
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = fmaf(a, static_cast<float>((lo >> (8 * k)) & 0xFFu), b);
      w[4 + k] = fmaf(a, static_cast<float>((hi >> (8 * k)) & 0xFFu), b);
    }
  } else {
    uint32_t ev = c.q0 & 0x0F0F0F0Fu, od = (c.q0 >> 4) & 0x0F0F0F0Fu;  // codes 0, 2, 4, 6 and 1, 3, 5, 7
    if constexpr (is_fifth(FMT)) {
      ev |= ((c.qh >> (2 * i)) & 0x01010101u) << 4;
      od |= ((c.qh >> (2 * i + 1)) & 0x01010101u) << 4;
    } else if constexpr (FMT == QMV_Q6K) {
      ev |= ((c.qh >> (4 * (i & 1))) & 0x03030303u) << 4;
      od |= ((c.qh >> (4 * (i & 1) + 2)) & 0x03030303u) << 4;
    }
    // whole bytes, as the conversion takes them: seeing the mask, the compiler
    // extracts four bits at a time instead (6 more instructions per 8 weights;
    // W4A16, 5632 x 2048, 512 tokens 36.5 against 34.0 us)
    asm("" : "+v"(ev), "+v"(od));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[2 * k] = fmaf(a, static_cast<float>((ev >> (8 * k)) & 0xFFu), b);
      w[2 * k + 1] = fmaf(a, static_cast<float>((od >> (8 * k)) & 0xFFu), b);
    }
  }
}

// One unit (32 weights of one row), as loaded.
template <int FMT>
struct UnitRaw {
  static constexpr int NQ = FMT == QMV_DENSE_BF16 ? 4 : is_byte(FMT) ? 2 : 1;
  u32x4 q[NQ];
  u32x2 qh;
  MetaRaw<FMT> m;
};

// Unit u of row r.
template <int FMT, By BY>
__device__ __forceinline__ UnitRaw<FMT> load_unit(const Mat& w, uint32_t row, int u, int K) {
  UnitRaw<FMT> x;
  constexpr int NQ = UnitRaw<FMT>::NQ;
  const RowAt<FMT> r = row_at<FMT>(row, K);
#pragma unroll
  for (int i = 0; i < NQ; ++i) x.q[i] = load_at<u32x4, BY>(w.p[0], r.o[0], int64_t(u) * (16 * NQ) + 16 * i);
  if constexpr (is_fifth(FMT)) x.qh[0] = load_at<uint32_t, BY>(w.p[1], r.o[1], 4 * u);
  if constexpr (FMT == QMV_Q6K) x.qh = load_at<u32x2, BY>(w.p[1], r.o[1], 8 * u);
  x.m = load_meta<FMT, BY>(w, r, u);
  return x;
}

// Word i (0..3) of a unit: its eight weights as one 16-byte piece.
template <int FMT, bool F16>
__device__ __forceinline__ u32x4 unit_piece(const UnitRaw<FMT>& r, const Affine& f, int i) {
  if constexpr (FMT == QMV_DENSE_BF16) {
    if constexpr (!F16) return r.q[i];
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t v = r.q[i][e];
      o[e] = pack16<F16>(bf16_bits_to_f32(v & 0xFFFFu), bf16_bits_to_f32(v >> 16));
    }
    return o;
  } else {
    Word8 c;
    if constexpr (is_byte(FMT)) {
      c.q0 = r.q[i >> 1][2 * (i & 1)];
      c.q1 = r.q[i >> 1][2 * (i & 1) + 1];
    } else {
      c.q0 = r.q[0][i];
    }
    if constexpr (is_fifth(FMT)) c.qh = r.qh[0];
    if constexpr (FMT == QMV_Q6K) c.qh = r.qh[i >> 1];
    float w[8];
    const bool second = FMT == QMV_Q6K && i >= 2;
    decode8<FMT>(c, second ? f.a1 : f.a0, second ? f.b1 : f.b0, i, w);
    return u32x4{pack16<F16>(w[0], w[1]), pack16<F16>(w[2], w[3]), pack16<F16>(w[4], w[5]), pack16<F16>(w[6], w[7])};
  }
}

// Half a unit: words 2 h and 2 h + 1 (16 weights).  The codes of kChunk
// consecutive units of a row are 64 bytes, which go to LDS as they are (a line
// is then fetched once, by four neighbouring lanes; one unit per step and lane
// instead fetched each 128-byte line four times, and its scales' line 32 times:
// 222 us of loads alone under 162 us of MFMA).  The scales of kRun units are
// loaded together.
template <int FMT>
constexpr int kChunk = FMT == QMV_DENSE_BF16 ? 1 : is_byte(FMT) ? 2 : 4;
constexpr int kRun = 8;

template <int FMT>
struct HalfRaw {
  u32x4 q[2];  // codes: two dwords; 8-bit: four; dense: eight
  uint32_t qh;
  MetaRaw<FMT> m;
};

// A tile of 64-byte rows of codes: WPT words (2: half w / 2; 1: word w) of unit s
// of row r, 0 <= s < kChunk.
template <int FMT, int WPT>
__device__ __forceinline__ void read_codes(u32x4 (&q)[2], const u32x4* R, int r, int s, int w) {
  if constexpr (FMT == QMV_DENSE_BF16) {
    q[0] = R[tile32_at(r, w)];
    if constexpr (WPT == 2) q[1] = R[tile32_at(r, w + 1)];
  } else if constexpr (is_byte(FMT)) {
    if constexpr (WPT == 2) {
      q[0] = R[tile32_at(r, 2 * s + (w >> 1))];
    } else {
      const u32x2 v = reinterpret_cast<const u32x2*>(R + tile32_at(r, 2 * s + (w >> 1)))[w & 1];
      q[0][0] = v[0];
      q[0][1] = v[1];
    }
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(R + tile32_at(r, s)) + w;
    if constexpr (WPT == 2) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      q[0][0] = v[0];
      q[0][1] = v[1];
    } else {
      q[0][0] = *p;
    }
  }
}

// Half h (a lane's) of unit u (a lane's too if BY is kByUnit) of a row, from global memory.
template <int FMT, By BY>
__device__ __forceinline__ HalfRaw<FMT> load_half(const Mat& w, const RowAt<FMT>& r, int u, int h) {
  HalfRaw<FMT> x;
  constexpr int B = 32 / kChunk<FMT>;  // bytes of half a unit's codes
  const uint32_t at = r.o[0] + B * h;
  const int64_t ub = int64_t(u) * (2 * B);
  if constexpr (B == 8) {
    const u32x2 v = load_at<u32x2, BY>(w.p[0], at, ub);
    x.q[0][0] = v[0];
    x.q[0][1] = v[1];
  } else {
    x.q[0] = load_at<u32x4, BY>(w.p[0], at, ub);
    if constexpr (B == 32) x.q[1] = load_at<u32x4, BY>(w.p[0], at, ub + 16);
  }
  if constexpr (is_fifth(FMT)) x.qh = load_at<uint32_t, BY>(w.p[1], r.o[1], 4 * u);
  if constexpr (FMT == QMV_Q6K) x.qh = load_at<uint32_t, BY>(w.p[1], r.o[1] + 4 * h, 8 * u);
  x.m = load_meta<FMT, BY>(w, r, u);
  return x;
}

// Makes the weights of r zeros unless `keep`: with a scale of zero every format
// gives zeros, whatever its codes.
template <int FMT>
__device__ __forceinline__ void keep_weights(HalfRaw<FMT>& r, bool keep) {
  if constexpr (FMT == QMV_DENSE_BF16) {
    const u32x4 zero = {0, 0, 0, 0};
    r.q[0] = keep ? r.q[0] : zero;
    r.q[1] = keep ? r.q[1] : zero;
  } else {
    constexpr int i = FMT == QMV_Q6K ? 1 : 0;  // the factor of all others
    r.m.v[i] = keep ? r.m.v[i] : 0u;
  }
}

// Word w of unit u as one 16-byte piece; its codes are the i-th of r.
template <int FMT, bool F16>
__device__ __forceinline__ u32x4 word_piece(const HalfRaw<FMT>& r, int u, int w, int i) {
  if constexpr (FMT == QMV_DENSE_BF16) {
    if constexpr (!F16) return r.q[i];
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t v = r.q[i][e];
      o[e] = pack16<F16>(bf16_bits_to_f32(v & 0xFFFFu), bf16_bits_to_f32(v >> 16));
    }
    return o;
  } else {
    Word8 c;
    if constexpr (is_byte(FMT)) {
      c.q0 = r.q[0][2 * i];
      c.q1 = r.q[0][2 * i + 1];
    } else {
      c.q0 = r.q[0][i];
    }
    c.qh = r.qh;
    const Affine f = affine_of<FMT>(r.m, u);
    float v[8];
    const bool second = FMT == QMV_Q6K && w >= 2;  // the second sub-block
    decode8<FMT>(c, second ? f.a1 : f.a0, second ? f.b1 : f.b0, w, v);
    return u32x4{pack16<F16>(v[0], v[1]), pack16<F16>(v[2], v[3]), pack16<F16>(v[4], v[5]), pack16<F16>(v[6], v[7])};
  }
}

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

// The scales and high bits of a run, for half h.
template <int FMT>
struct RunMeta {
  uint32_t qh[8];
  u32x4 m;
  uint32_t d;
};

// Loads of load_run_meta, at least.
template <int FMT>
constexpr int kMetaLoads = FMT == QMV_DENSE_BF16 ? 0 : is_fifth(FMT) ? 3 : FMT == QMV_Q6K ? 10 : 1;

// Units u .. u + kRun - 1 of row r; u is a multiple of kRun and the run is
// inside the row.
template <int FMT>
__device__ __forceinline__ RunMeta<FMT> load_run_meta(const Mat& w, uint32_t r, int u, int h, int K) {
  RunMeta<FMT> x;
  constexpr int S = kRun, P = kPlanes<FMT> - 1;
  const uint32_t mt = r * row_bytes<FMT>(P, K), ht = r * row_bytes<FMT>(1, K);
  if constexpr (is_fifth(FMT)) {
    const u32x4 a = load_at<u32x4_a4, kByRow>(w.p[1], ht, 4 * u), b = load_at<u32x4_a4, kByRow>(w.p[1], ht, 4 * u + 16);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      x.qh[s] = a[s];
      x.qh[4 + s] = b[s];
    }
  }
  if constexpr (FMT == QMV_Q8_0 || FMT == QMV_Q4_0 || FMT == QMV_Q5_0) {
    x.m = load_at<u32x4_a2, kByRow>(w.p[P], mt, 2 * u);
  } else if constexpr (FMT == QMV_W4A16_G64) {
    x.m = load_at<u32x4_a4, kByRow>(w.p[P], mt, 2 * u);
  } else if constexpr (is_super(FMT)) {
    x.m = load_at<u32x4, kByRow>(w.p[P], mt, 16 * (u >> 3));
  } else if constexpr (FMT == QMV_Q6K) {
#pragma unroll
    for (int s = 0; s < S; ++s) x.qh[s] = load_at<uint32_t, kByRow>(w.p[1], ht + 4 * h, 8 * (u + s));
    x.m = load_at<u32x4, kByRow>(w.p[2], r * row_bytes<FMT>(2, K), 2 * u);
    x.d = load_at<uint16_t, kByRow>(w.p[3], mt, 2 * (u >> 3));
  } else if constexpr (FMT == QMV_I8_ROW) {
    x.m[0] = load_at<uint32_t, kByRow>(w.p[1], mt);
  }
  return x;
}

// The scales of unit u + s of a run (s known at compile time).
template <int FMT>
__device__ __forceinline__ void meta_of(HalfRaw<FMT>& r, const RunMeta<FMT>& x, int s) {
  r.qh = x.qh[s];
  if constexpr (FMT == QMV_Q6K || FMT == QMV_Q8_0 || FMT == QMV_Q4_0 || FMT == QMV_Q5_0) {
    r.m.v[0] = (x.m[s >> 1] >> (16 * (s & 1))) & 0xFFFFu;
    r.m.v[1] = x.d;
  } else if constexpr (FMT == QMV_W4A16_G64) {
    r.m.v[0] = x.m[s >> 1];
  } else {
    r.m.v = x.m;
  }
}

// 16 bytes from global memory (buffer base + lane offset + uniform offset)
// straight into LDS: the wave's 64 pieces land at `dst` (uniform) in lane order.
// A buffer instruction, because the global_load_lds form counts as a flat access
// with the compiler, which then lets every later wait drain both counters.
typedef __amdgpu_buffer_rsrc_t Buf;
__device__ __forceinline__ Buf buffer_of(const void* base, int bytes = -1) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ Buf buffer_of(const QMV_GLOBAL uint8_t* base, int bytes = -1) {
  return buffer_of((const void*)base, bytes);
}
__device__ __forceinline__ void copy_to_lds(Buf b, uint32_t lane, uint32_t uniform, u32x4* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (void __attribute__((address_space(3)))*)dst, 16, lane, uniform, 0, 0);
}

// ---------------------------------------------------------------- activations
// act(g), and act'(g) for the backward pass.  exp and reciprocal are the
// hardware's (about 1 ulp in f32), far below the 16-bit rounding of the result.
__device__ __forceinline__ float sigmoid16(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

__device__ __forceinline__ float gelu_tanh_arg(float g) {  // 2 sqrt(2/pi) (g + 0.044715 g^3): (1 + tanh(z)) / 2 = sigmoid(2 z)
  const float c = fminf(fmaxf(g, -20.0f), 20.0f);  // saturated far before 20: keeps g^3 finite
  return 1.5957691216057308f * fmaf(0.044715f * c * c, c, c);
}

// (1 + erf(g / sqrt 2)) / 2, and e = exp(-g^2 / 2).  With z = |g| / sqrt 2 and
// t = 1 / (1 + z / 2), erfc(z) exp(z^2) = t Q(t); the coefficients are those of
// Q / 2, fitted to the smallest largest relative error over z in [0, 11] (4e-8;
// exp is zero past it).  In f32 the whole is within 7e-7 for |g| <= 3 and 4e-6 for
// |g| <= 9, which is what one rounding of g changes there (the relative slope is
// g).  The library's erfc, some three times the instructions, cost 1 us more in
// an epilogue of 16 values per thread.
__device__ __forceinline__ float normal_cdf(float g, float& e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(g), 0.35355339f, 1.0f));
  float q = -0.0296387542f;
  q = fmaf(q, t, 0.142796725f);
  q = fmaf(q, t, -0.244655371f);
  q = fmaf(q, t, 0.14024204f);
  q = fmaf(q, t, -0.0141459107f);
  q = fmaf(q, t, 0.101696089f);
  q = fmaf(q, t, 0.12146274f);
  q = fmaf(q, t, 0.141199902f);
  q = fmaf(q, t, 0.141042516f);
  e = __builtin_amdgcn_exp2f(g * g * -0.72134752f);
  const float p = q * t * e;
  return g < 0.0f ? p : 1.0f - p;
}

// The activation is a template argument where many values go through one
// (as a runtime choice every value paid for all three: 16 us per workgroup of
// 256 x 128 outputs).
template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == QMV_ACT_SILU) {
    return g * sigmoid16(g);
  } else if constexpr (ACT == QMV_ACT_GELU_TANH) {
    return g * sigmoid16(gelu_tanh_arg(g));
  } else {
    float e;
    return g * normal_cdf(g, e);
  }
}

__device__ __forceinline__ float act_of(int act, float g) {
  return act == QMV_ACT_SILU ? act_value<QMV_ACT_SILU>(g)
         : act == QMV_ACT_GELU_TANH ? act_value<QMV_ACT_GELU_TANH>(g) : act_value<QMV_ACT_GELU>(g);
}

template <int ACT>
__device__ __forceinline__ void act_both(float g, float& a, float& da) {
  if constexpr (ACT == QMV_ACT_SILU) {
    const float s = sigmoid16(g);
    a = g * s;
    da = s * fmaf(g, 1.0f - s, 1.0f);
  } else if constexpr (ACT == QMV_ACT_GELU_TANH) {
    const float s = sigmoid16(gelu_tanh_arg(g));
    const float c = fminf(fmaxf(g, -20.0f), 20.0f);
    a = g * s;
    da = fmaf(g * s, (1.0f - s) * 1.5957691216057308f * fmaf(0.134145f * c, c, 1.0f), s);
  } else {
    float e;
    const float p = normal_cdf(g, e);
    a = g * p;
    da = fmaf(g, 0.3989422804014327f * e, p);
  }
}

}  // namespace qmv
