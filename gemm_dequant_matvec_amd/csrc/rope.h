// Shared by the rotary positions (rope.hip) and the normed heads with rotary
// positions (norm_rope.hip): the sine and cosine of a far position, and pieces
// of heads between memory and f32 registers.
//
// The angle of a far position needs more than f64 gives to a product: pos * freq
// has 31 + 24 bits.  It is kept as a rounded product and what the rounding left
// over, turned into revolutions by a 1 / (2 pi) of two parts, and reduced to an
// eighth of a turn, all in f64.  For f32 heads sin and cos are Taylor polynomials in
// f64 (degree 13 and 12: truncation below 1e-12 on [-pi/4, pi/4]), and what a pair is
// multiplied by, amplitude included, is rounded to f32 once.  For 16-bit heads the
// reduced angle is rounded to f32 and the polynomials are f32 (degree 11 and 10,
// below 1e-9): 2^-22 against the 2^-12 of their own rounding, and the f64 ones take
// longer than the bytes there (4096 tokens 11.0 against 8.9 us, bf16).
#pragma once

#include "gemm16.h"

namespace qmv {
namespace {

// amplitude cos(pos freq) and amplitude sin(pos freq); WIDE: rounded to f32 once.
template <bool WIDE>
__device__ __forceinline__ void turn(int64_t pos, float freq, float amplitude, float& c, float& s) {
#pragma clang fp contract(off)  // a product must be rounded where its rest is taken
  const double a = double(pos), f = double(freq);
  const double t = a * f, t_low = fma(a, f, -t);  // a f = t + t_low
  constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;  // 1 / (2 pi)
  const double rev = t * kInv;
  const double low = fma(t, kInv, -rev) + fma(t, kInvLow, t_low * kInv);
  const double r = (rev - rint(rev)) + low;  // [-1/2, 1/2], off by less than 2^-52
  const double q = rint(4.0 * r);
  const double y = (r - 0.25 * q) * 6.283185307179586;  // [-pi/4, pi/4]
  const int n = int(q) & 3;  // quarter turns
  float sp, cp;
  if constexpr (WIDE) {
    const double z = y * y;
    double sd = 1.0 / 6227020800, cd = 1.0 / 479001600;  // 1 / 13!, 1 / 12!
    sd = fma(z, sd, -1.0 / 39916800);
    cd = fma(z, cd, -1.0 / 3628800);
    sd = fma(z, sd, 1.0 / 362880);
    cd = fma(z, cd, 1.0 / 40320);
    sd = fma(z, sd, -1.0 / 5040);
    cd = fma(z, cd, -1.0 / 720);
    sd = fma(z, sd, 1.0 / 120);
    cd = fma(z, cd, 1.0 / 24);
    sd = fma(z, sd, -1.0 / 6);
    cd = fma(z, cd, -1.0 / 2);
    sp = float(amplitude * (y * fma(z, sd, 1.0)));
    cp = float(amplitude * fma(z, cd, 1.0));
  } else {
    const float yf = float(y), z = yf * yf;
    sp = yf * fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.50521084e-8f, 2.75573192e-6f), -1.98412698e-4f),
                                   8.33333333e-3f), -1.66666667e-1f), 1.0f);
    cp = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.75573192e-7f, 2.48015873e-5f), -1.38888889e-3f),
                              4.16666667e-2f), -0.5f), 1.0f);
    sp *= amplitude;
    cp *= amplitude;
  }
  c = n == 0 ? cp : n == 1 ? -sp : n == 2 ? -cp : sp;
  s = n == 0 ? sp : n == 1 ? cp : n == 2 ? -sp : -cp;
}

template <int E>  // 0: f32, 1: f16, 2: bf16
struct Elem {
  static constexpr int V = E == 0 ? 4 : 8;  // values per 16 bytes
  typedef typename std::conditional<E == 0, float, uint16_t>::type T;
  static __device__ __forceinline__ float get(T v) {
    if constexpr (E == 0) return v;
    else return unpack16<E == 1>(v);
  }
  static __device__ __forceinline__ T put(float v) {
    if constexpr (E == 0) return v;
    else return uint16_t(pack16<E == 1>(v, 0.f));
  }
  // n (1 .. V) values from p as they are, zeros behind them; the whole vector in one load
  static __device__ __forceinline__ u32x4 raw(const T* p, int n) {
    u32x4 w = {0, 0, 0, 0};
    if (n == V) {
      __builtin_memcpy(&w, p, 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) {
          if constexpr (E == 0) w[i] = __builtin_bit_cast(uint32_t, p[i]);
          else w[i >> 1] |= uint32_t(p[i]) << (16 * (i & 1));
        }
    }
    return w;
  }
  static __device__ __forceinline__ void values(u32x4 w, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = w[i];
      if constexpr (E == 0) {
        v[i] = __builtin_bit_cast(float, b);
      } else {
        v[2 * i] = unpack16<E == 1>(b & 0xFFFFu);
        v[2 * i + 1] = unpack16<E == 1>(b >> 16);
      }
    }
  }
  // the same in f32
  static __device__ __forceinline__ void load(const T* p, int n, float (&v)[V]) { values(raw(p, n), v); }
  static __device__ __forceinline__ void store(T* p, int n, const float (&v)[V]) {
    if (n == V) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (E == 0) w[i] = __builtin_bit_cast(uint32_t, v[i]);
        else w[i] = pack16<E == 1>(v[2 * i], v[2 * i + 1]);
      }
      __builtin_memcpy(p, &w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) p[i] = put(v[i]);
    }
  }
};

}  // namespace
}  // namespace qmv
