// Rotary positions of the q and k heads.
//
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t), t = pos * freq_i
//
// for the pairs (x_i, x_{i + R/2}) (half) or (x_2i, x_2i+1) (interleaved) of the
// first R values of every head; the other D - R values pass.  The inverse
// (t -> -t) is the gradient.  Bound by memory: each value is read and written
// once, so a block computes the R/2 sines and cosines of its tokens once, into
// LDS, for all heads of all tensors.  A block takes tokens up to about 16 KB of
// heads, so that its threads have several 16-byte pieces each and the sines are
// not the longer part, but no more than leave 512 blocks.  f16, 24 heads of 128,
// 32768 tokens: 81 us, 4.95 TB/s (a copy of 1 GiB runs at 5.1); bf16, 36 heads of
// 64, 4096 tokens: 8.8 us, 4.3 TB/s; one token (f32) 3.0 us, the launch.
// Far positions: rope.h.
#include <algorithm>
#include <cmath>

#include "rope.h"

namespace qmv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 2048;  // cosine / sine pairs a block keeps (16 KB)

struct RopeTensor {
  const void* x;
  void* y;
  int64_t xt, xh, yt, yh;  // strides of token and head, in elements
  int heads, copy;         // copy: the values past R have to be written too
};
struct RopeArgs {
  RopeTensor t[QMV_ROPE_MAX];
  int count, D, R, tb;     // tb: tokens per block
  int64_t T;
  const int64_t* pos;
  const float* freqs;
  float amplitude, sign;
};

template <int E, bool HALF>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs p) {
  typedef Elem<E> El;
  typedef typename El::T T;
  constexpr int V = El::V;
  __shared__ float2 cs[kMaxPairs];
  const int tid = threadIdx.x;
  const int P = p.R >> 1;
  // pieces of a head: the rotated ones, then the passing ones
  const int nr = HALF ? (P + V - 1) / V : (p.R + V - 1) / V;
  for (int64_t t0 = int64_t(blockIdx.x) * p.tb; t0 < p.T; t0 += int64_t(gridDim.x) * p.tb) {
    const int nt = int(min(int64_t(p.tb), p.T - t0));
    for (int i = tid; i < nt * P; i += kThreads) {
      const int t = i / P, f = i - t * P;
      float c, s;
      turn<E == 0>(p.pos[t0 + t], p.freqs[f], p.amplitude, c, s);
      cs[i] = make_float2(c, p.sign * s);
    }
    __syncthreads();

#pragma unroll 1
    for (int k = 0; k < p.count; ++k) {
      const RopeTensor& q = p.t[k];
      const int np = nr + (q.copy ? (p.D - p.R + V - 1) / V : 0);
      const int items = nt * q.heads * np;
      for (int it = tid; it < items; it += kThreads) {
        const int th = it / np, c = it - th * np;
        const int t = th / q.heads, h = th - t * q.heads;
        const T* x = static_cast<const T*>(q.x) + (t0 + t) * q.xt + h * q.xh;
        T* y = static_cast<T*>(q.y) + (t0 + t) * q.yt + h * q.yh;
        if (c >= nr) {
          const int at = p.R + (c - nr) * V, n = min(V, p.D - at);
          float v[V];
          El::load(x + at, n, v);
          El::store(y + at, n, v);
        } else if constexpr (HALF) {
          const int i0 = c * V, n = min(V, P - i0);
          float a[V], b[V];
          El::load(x + i0, n, a);
          El::load(x + P + i0, n, b);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 w = cs[t * P + min(i0 + i, P - 1)];
            const float u = a[i];
            a[i] = fmaf(-b[i], w.y, u * w.x);
            b[i] = fmaf(u, w.y, b[i] * w.x);
          }
          El::store(y + i0, n, a);
          El::store(y + P + i0, n, b);
        } else {
          const int i0 = c * V, n = min(V, p.R - i0);
          float a[V];
          El::load(x + i0, n, a);
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float2 w = cs[t * P + min((i0 + i) >> 1, P - 1)];
            const float u = a[i];
            a[i] = fmaf(-a[i + 1], w.y, u * w.x);
            a[i + 1] = fmaf(u, w.y, a[i + 1] * w.x);
          }
          El::store(y + i0, n, a);
        }
      }
    }
    __syncthreads();  // the sines of these tokens are done with
  }
}

}  // namespace

hipError_t launch_rope(int64_t T, int D, int R, int layout, int count, const qmv_rope_tensor* t, int dtype,
                       const int64_t* pos, const float* freqs, float amplitude, int inverse, hipStream_t s) {
  RopeArgs p{};
  int heads = 0;
  for (int i = 0; i < count; ++i) {
    p.t[i] = RopeTensor{t[i].x, t[i].y, t[i].x_token, t[i].x_head, t[i].y_token, t[i].y_head, int(t[i].heads),
                        t[i].x != t[i].y};
    heads += int(t[i].heads);
  }
  p.count = count;
  p.D = D;
  p.R = R;
  p.T = T;
  p.pos = pos;
  p.freqs = freqs;
  p.amplitude = amplitude;
  p.sign = inverse ? -1.0f : 1.0f;
  const int per = heads * D * (dtype == QMV_F32 ? 4 : 2);  // bytes of a token
  int64_t tb = std::max(1, 16384 / per);
  tb = std::min<int64_t>({tb, std::max<int64_t>(1, kMaxPairs / (R / 2)), std::max<int64_t>(1, T / 512)});
  p.tb = int(tb);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((T + tb - 1) / tb, 1 << 20)));
  const bool half = layout == QMV_ROPE_HALF;
#define QMV_ROPE_GO(E)                                                                   \
  if (half) hipLaunchKernelGGL((rope_kernel<E, true>), grid, dim3(kThreads), 0, s, p);   \
  else hipLaunchKernelGGL((rope_kernel<E, false>), grid, dim3(kThreads), 0, s, p);
  if (dtype == QMV_F32) {
    QMV_ROPE_GO(0)
  } else if (dtype == QMV_F16) {
    QMV_ROPE_GO(1)
  } else {
    QMV_ROPE_GO(2)
  }
#undef QMV_ROPE_GO
  return hipGetLastError();
}

}  // namespace qmv
