// Norms of the q and k heads with their rotary positions, and the gradient.
//
//   r = (mean(x^2) + eps)^(-1/2),  n = x r,  y = rot(n (w + offset))
//   g = rot^T(dy),  h = g (w + offset),  dx = r (h - n mean(h n)),  dw = sum of g n
//
// over the D values of a head; rot as in rope.hip.  Bound by memory: x (and dy)
// are read once, y (dx) is written once.  A head belongs to a group of L lanes of
// one wave, L the power of two that holds its 16-byte pieces (pairs of pieces, x_i
// and x_{i + R/2}, in the half layout, so that a rotary pair is in one lane); the
// sums over a head are L-lane sums of registers, and a lane's weights, the same for
// every head that it takes, stay in registers.  A block works on one tensor (q or
// k) and computes the sines of its tokens once, into LDS.  Forward, a head is under
// way while the sines or the head before it are worked on: 16384 tokens of 32 + 8
// heads of 128, bf16, 103 -> 88 us, with no more blocks than the chip holds 67 (5.0
// TB/s; a copy reaches 5.1).  Backward the registers that this takes cost more than
// it gives (108 us without, 4.7 TB/s, of which the second launch 5; 20 more with).
//
// The weights' gradient: a lane sums g n over its heads in f32, the lanes of a wave
// and the waves of a block that hold the same values are added in a fixed order, a
// block's sums go to the workspace, and a second launch adds the blocks', in a fixed
// order too: no atomics, calls repeat bit for bit.
#include <algorithm>

#include "rope.h"

namespace qmv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 2048;  // cosine / sine pairs a block keeps (16 KB)

struct NormTensor {
  const void* x;
  const void* dy;  // backward
  void* y;         // forward: y, backward: dx
  const void* w;   // NULL: 1
  float* part;     // backward: [blocks][D] partial sums of dw; NULL: dw is not wanted
  int64_t xt, xh, gt, gh, yt, yh;  // strides of token and head, in elements
  int heads, tb, first, blocks;    // tokens per turn of a block, first block, blocks
};
struct NormArgs {
  NormTensor t[QMV_ROPE_MAX];
  int count, D, R, L, w_f32;
  int64_t T;
  const int64_t* pos;
  const float* freqs;
  float amplitude, eps, offset;
};

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// Sum over a group of L lanes (a power of two), in every lane of it.
__device__ __forceinline__ float group_sum(float v, int L) {
  if (L > 1) v = dpp_add<0xB1>(v);   // lane ^ 1
  if (L > 2) v = dpp_add<0x4E>(v);   // lane ^ 2
  if (L > 4) v = dpp_add<0x141>(v);  // mirrored in 8 lanes: the other four
  if (L > 8) v = dpp_add<0x140>(v);  // mirrored in 16 lanes: the other eight
  if (L > 16) v += __shfl_xor(v, 16);
  if (L > 32) v += __shfl_xor(v, 32);
  return v;
}

// The pieces of a head that a lane holds: J pieces a[j], with the second halves of
// their pairs b[j] in the half layout.
template <int E, bool HALF, int J>
struct Pieces {
  typedef Elem<E> El;
  typedef typename El::T T;
  static constexpr int V = El::V;
  int at[J], n[J];    // first value of a[j] and how many (0: none)
  int bt[J], bn[J];   // the same for b[j]
  int angle[J];       // index of the first pair's sine, -1: the values pass

  __device__ __forceinline__ void init(int lane, int L, int D, int R) {
    const int P = R >> 1, nr = HALF ? (P + V - 1) / V : (R + V - 1) / V;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = lane + j * L;
      const bool turned = c < nr;
      at[j] = turned ? c * V : R + (c - nr) * V;
      n[j] = max(0, min(V, (turned ? (HALF ? P : R) : D) - at[j]));
      angle[j] = !turned ? -1 : HALF ? c * V : c * V / 2;
      bt[j] = P + c * V;
      bn[j] = HALF && turned ? n[j] : 0;
    }
  }
  struct Raw {  // as they are in memory
    u32x4 a[J], b[J];
    __device__ __forceinline__ void values(float (&x)[J][V], float (&y)[J][V]) const {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        El::values(a[j], x[j]);
        if constexpr (HALF) El::values(b[j], y[j]);
      }
    }
  };
  __device__ __forceinline__ void load(const T* p, Raw& r) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      r.a[j] = El::raw(p + at[j], n[j]);
      if constexpr (HALF) r.b[j] = El::raw(p + bt[j], bn[j]);
    }
  }
  __device__ __forceinline__ void store(T* p, const float (&a)[J][V], const float (&b)[J][V]) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      El::store(p + at[j], n[j], a[j]);
      if constexpr (HALF) El::store(p + bt[j], bn[j], b[j]);
    }
  }
  // the weights of these places, w + offset; 1 without weights
  __device__ __forceinline__ void weights(const void* w, int f32, float offset, float (&a)[J][V], float (&b)[J][V]) const {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[j][i] = i < n[j] ? weight(w, f32, offset, at[j] + i) : 0.0f;
        if constexpr (HALF) b[j][i] = i < bn[j] ? weight(w, f32, offset, bt[j] + i) : 0.0f;
      }
  }
  static __device__ __forceinline__ float weight(const void* w, int f32, float offset, int i) {
    if (!w) return 1.0f;
    return (f32 ? static_cast<const float*>(w)[i] : El::get(static_cast<const T*>(w)[i])) + offset;
  }
  // cs: the cosines and sines of the head's token, P of them
  __device__ __forceinline__ void rotate(const float2* cs, int P, float (&a)[J][V], float (&b)[J][V]) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (angle[j] < 0) continue;
      if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 w = cs[min(angle[j] + i, P - 1)];
          const float u = a[j][i];
          a[j][i] = fmaf(-b[j][i], w.y, u * w.x);
          b[j][i] = fmaf(u, w.y, b[j][i] * w.x);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 w = cs[min(angle[j] + (i >> 1), P - 1)];
          const float u = a[j][i];
          a[j][i] = fmaf(-a[j][i + 1], w.y, u * w.x);
          a[j][i + 1] = fmaf(u, w.y, a[j][i + 1] * w.x);
        }
      }
    }
  }
};

template <int E>
__device__ __forceinline__ void fill_sines(const NormArgs& p, float sign, int64_t t0, int nt, float2* cs) {
  const int P = p.R >> 1;
  for (int i = threadIdx.x; i < nt * P; i += kThreads) {
    const int t = i / P, f = i - t * P;
    float c, s;
    turn<E == 0>(p.pos[t0 + t], p.freqs[f], p.amplitude, c, s);
    cs[i] = make_float2(c, sign * s);
  }
}

__device__ __forceinline__ int tensor_of_block(const NormArgs& p) {
  int k = 0;
  while (k + 1 < p.count && int(blockIdx.x) >= p.t[k + 1].first) ++k;
  return k;
}

// The heads that a group of lanes takes of a turn's tokens: every `groups`-th one.
struct Place {
  int t, h, left;  // token of the turn, head, heads from this one to the turn's last
  int heads, dt, dh, groups;
  __device__ __forceinline__ Place(int heads, int groups) : heads(heads), groups(groups) {
    dt = groups / heads;
    dh = groups - dt * heads;
  }
  __device__ __forceinline__ void start(int group, int tokens) {
    t = group / heads;
    h = group - t * heads;
    left = tokens * heads - group;
  }
  __device__ __forceinline__ bool any() const { return left > 0; }
  __device__ __forceinline__ void next() {
    t += dt;
    h += dh;
    if (h >= heads) h -= heads, ++t;
    left -= groups;
  }
};

template <int E, bool HALF, int J>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(const NormArgs p) {
  typedef Pieces<E, HALF, J> Pc;
  typedef typename Pc::T T;
  constexpr int V = Pc::V;
  extern __shared__ float2 cs[];
  const NormTensor& q = p.t[tensor_of_block(p)];
  const int L = p.L, P = p.R >> 1, groups = kThreads / L, group = threadIdx.x / L;
  Pc pc;
  pc.init(threadIdx.x & (L - 1), L, p.D, p.R);
  Place at(q.heads, groups);
  typename Pc::Raw raw;
  float wa[J][V], wb[J][V];
  const T* const x = static_cast<const T*>(q.x);
  int64_t t0 = int64_t(blockIdx.x - q.first) * q.tb;
  at.start(group, int(min(int64_t(q.tb), p.T - t0)));
  if (at.any()) pc.load(x + (t0 + at.t) * q.xt + at.h * q.xh, raw);  // the first heads come while the sines are made
  pc.weights(q.w, p.w_f32, p.offset, wa, wb);
  for (; t0 < p.T; t0 += int64_t(q.blocks) * q.tb) {
    fill_sines<E>(p, 1.0f, t0, int(min(int64_t(q.tb), p.T - t0)), cs);
    __syncthreads();
    while (at.any()) {
      const int t = at.t;
      T* const y = static_cast<T*>(q.y) + (t0 + t) * q.yt + at.h * q.yh;
      float a[J][V], b[J][V], ss = 0.0f;
      raw.values(a, b);
      at.next();
      if (at.any()) pc.load(x + (t0 + at.t) * q.xt + at.h * q.xh, raw);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          ss = fmaf(a[j][i], a[j][i], ss);
          if constexpr (HALF) ss = fmaf(b[j][i], b[j][i], ss);
        }
      const float r = 1.0f / sqrtf(group_sum(ss, L) / float(p.D) + p.eps);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          a[j][i] = a[j][i] * r * wa[j][i];
          if constexpr (HALF) b[j][i] = b[j][i] * r * wb[j][i];
        }
      pc.rotate(cs + t * P, P, a, b);
      pc.store(y, a, b);
    }
    const int64_t n0 = t0 + int64_t(q.blocks) * q.tb;
    if (n0 >= p.T) break;
    at.start(group, int(min(int64_t(q.tb), p.T - n0)));
    if (at.any()) pc.load(x + (n0 + at.t) * q.xt + at.h * q.xh, raw);
    __syncthreads();  // the sines of these tokens are done with
  }
}

template <int E, bool HALF, int J>
__global__ __launch_bounds__(kThreads) void norm_rope_backward_kernel(const NormArgs p) {
  typedef Pieces<E, HALF, J> Pc;
  typedef typename Pc::T T;
  constexpr int V = Pc::V;
  extern __shared__ float2 cs[];  // and, at the end, [4 waves][D] sums
  const NormTensor& q = p.t[tensor_of_block(p)];
  const int L = p.L, P = p.R >> 1, groups = kThreads / L, group = threadIdx.x / L;
  Pc pc;
  pc.init(threadIdx.x & (L - 1), L, p.D, p.R);
  float wa[J][V], wb[J][V], sa[J][V], sb[J][V];
  pc.weights(q.w, p.w_f32, p.offset, wa, wb);
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) sa[j][i] = sb[j][i] = 0.0f;
  for (int64_t t0 = int64_t(blockIdx.x - q.first) * q.tb; t0 < p.T; t0 += int64_t(q.blocks) * q.tb) {
    const int nt = int(min(int64_t(q.tb), p.T - t0));
    fill_sines<E>(p, -1.0f, t0, nt, cs);
    __syncthreads();
    for (int it = group; it < nt * q.heads; it += groups) {
      const int t = it / q.heads, h = it - t * q.heads;
      float a[J][V], b[J][V], ga[J][V], gb[J][V], ss = 0.0f, hx = 0.0f;
      typename Pc::Raw rx, rg;
      pc.load(static_cast<const T*>(q.x) + (t0 + t) * q.xt + h * q.xh, rx);
      pc.load(static_cast<const T*>(q.dy) + (t0 + t) * q.gt + h * q.gh, rg);
      rx.values(a, b);
      rg.values(ga, gb);
      pc.rotate(cs + t * P, P, ga, gb);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          ss = fmaf(a[j][i], a[j][i], ss);
          hx = fmaf(ga[j][i] * wa[j][i], a[j][i], hx);
          if constexpr (HALF) {
            ss = fmaf(b[j][i], b[j][i], ss);
            hx = fmaf(gb[j][i] * wb[j][i], b[j][i], hx);
          }
        }
      const float r = 1.0f / sqrtf(group_sum(ss, L) / float(p.D) + p.eps);
      const float m = group_sum(hx, L) * r / float(p.D);  // mean(h n)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float n = a[j][i] * r;
          sa[j][i] = fmaf(ga[j][i], n, sa[j][i]);
          a[j][i] = r * fmaf(-n, m, ga[j][i] * wa[j][i]);
          if constexpr (HALF) {
            const float o = b[j][i] * r;
            sb[j][i] = fmaf(gb[j][i], o, sb[j][i]);
            b[j][i] = r * fmaf(-o, m, gb[j][i] * wb[j][i]);
          }
        }
      pc.store(static_cast<T*>(q.y) + (t0 + t) * q.yt + h * q.yh, a, b);
    }
    __syncthreads();  // the sines of these tokens are done with
  }
  if (!q.part) return;
  // the groups of a wave, then the waves of the block
  float* red = reinterpret_cast<float*>(cs);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      for (int s = L; s < 64; s <<= 1) {
        sa[j][i] += __shfl_xor(sa[j][i], s);
        if constexpr (HALF) sb[j][i] += __shfl_xor(sb[j][i], s);
      }
      if (lane < L) {
        if (i < pc.n[j]) red[wave * p.D + pc.at[j] + i] = sa[j][i];
        if constexpr (HALF)
          if (i < pc.bn[j]) red[wave * p.D + pc.bt[j] + i] = sb[j][i];
      }
    }
  __syncthreads();
  float* out = q.part + int64_t(blockIdx.x - q.first) * p.D;
  for (int d = threadIdx.x; d < p.D; d += kThreads)
    out[d] = (red[d] + red[p.D + d]) + (red[2 * p.D + d] + red[3 * p.D + d]);
}

// dw[d] = the sum over the blocks' partial sums, rounded once.  Block: 32 values d,
// 32 threads for each of them, with several of their loads under way.
struct SumArgs {
  struct {
    const float* part;
    void* dw;
    int blocks;
  } t[QMV_ROPE_MAX];
  int D, w_f32;
};
template <int E>
__global__ __launch_bounds__(1024) void norm_weight_kernel(const SumArgs p) {
  constexpr int kAhead = 16;
  __shared__ float red[32][33];
  const auto& q = p.t[blockIdx.y];
  if (!q.dw) return;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, d = blockIdx.x * 32 + x;
  float s = 0.0f;
  if (d < p.D)
    for (int b0 = y; b0 < q.blocks; b0 += 32 * kAhead) {
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v[i] = b0 + 32 * i < q.blocks ? q.part[int64_t(b0 + 32 * i) * p.D + d] : 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s += v[i];
    }
  red[y][x] = s;
  __syncthreads();
  for (int h = 16; h > 0; h >>= 1) {
    if (y < h) red[y][x] += red[y + h][x];
    __syncthreads();
  }
  if (y || d >= p.D) return;
  if (p.w_f32) static_cast<float*>(q.dw)[d] = red[0][x];
  else static_cast<typename Elem<E>::T*>(q.dw)[d] = Elem<E>::put(red[0][x]);
}

// Lanes of a group and pieces of a lane.
void shape_of(int D, int R, bool half, int dtype, int& L, int& J) {
  const int V = dtype == QMV_F32 ? 4 : 8, P = R / 2;
  const int np = (half ? (P + V - 1) / V : (R + V - 1) / V) + (D - R + V - 1) / V;
  for (L = 1; L < np && L < 64;) L <<= 1;
  J = (np + L - 1) / L;
}

template <class F>
void dispatch(int dtype, bool half, int J, F&& go) {
  auto with_j = [&](auto e, auto h) {
    if (J == 1) go(e, h, std::integral_constant<int, 1>{});
    else if (J == 2) go(e, h, std::integral_constant<int, 2>{});
    else go(e, h, std::integral_constant<int, 5>{});
  };
  auto with_h = [&](auto e) {
    if (half) with_j(e, std::true_type{});
    else with_j(e, std::false_type{});
  };
  if (dtype == QMV_F32) with_h(std::integral_constant<int, 0>{});
  else if (dtype == QMV_F16) with_h(std::integral_constant<int, 1>{});
  else with_h(std::integral_constant<int, 2>{});
}

NormArgs common(int64_t T, int D, int R, int count, int w_f32, const int64_t* pos, const float* freqs, float amplitude,
                float eps, float offset) {
  NormArgs p{};
  p.count = count;
  p.D = D;
  p.R = R;
  p.w_f32 = w_f32;
  p.T = T;
  p.pos = pos;
  p.freqs = freqs;
  p.amplitude = amplitude;
  p.eps = eps;
  p.offset = offset;
  return p;
}

}  // namespace

// One launch's worth of blocks, each with its turns: 16384 tokens of 32 + 8 heads of 128, bf16, half layout, take 67
// us with the 5 blocks that a unit holds, 71 with twice as many, 88 with one turn to a block; interleaved, 75 with 7 of the 8
// that it may hold, 89 with 8, 82 with one turn.  The tensors share them by heads and a token's sines, which cost about two.
constexpr int kSineHeads = 2;

// Tokens of a block's turn: the fewest, up to cap, whose heads fill the groups' last round to a few percent (35
// heads of 130, interleaved, f16, 11638 tokens: 118 us with one token, 98 with five).
int64_t tokens_of_turn(int64_t heads, int64_t groups, int64_t cap) {
  int64_t best = 1, best_rounds = (heads + groups - 1) / groups;
  for (int64_t tb = 1; tb <= cap; ++tb) {
    const int64_t rounds = (tb * heads + groups - 1) / groups;
    if (rounds * best < best_rounds * tb) best = tb, best_rounds = rounds;
    if (rounds * groups * 100 <= tb * heads * 103) break;
  }
  return best;
}

hipError_t launch_norm_rope(int64_t T, int D, int R, int layout, int count, const qmv_norm_rope_tensor* t, int dtype,
                            int w_dtype, float eps, float offset, const int64_t* pos, const float* freqs, float amplitude,
                            hipStream_t s) {
  NormArgs p = common(T, D, R, count, w_dtype == QMV_F32, pos, freqs, amplitude, eps, offset);
  int J;
  int64_t all = 0;
  for (int i = 0; i < count; ++i) all += t[i].heads + kSineHeads;
  shape_of(D, R, layout == QMV_ROPE_HALF, dtype, p.L, J);
  dispatch(dtype, layout == QMV_ROPE_HALF, J, [&](auto e, auto h, auto j) {
    auto kernel = norm_rope_kernel<decltype(e)::value, decltype(h)::value, decltype(j)::value>;
    static const int64_t resident = [&] {  // blocks of the whole chip
      int n = 0;
      if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, 0) != hipSuccess || n < 1) {
        (void)hipGetLastError();
        n = 4;
      }
      return int64_t(256) * std::min(n, 7);
    }();
    int first = 0, most = 1;
    for (int i = 0; i < count; ++i) {
      NormTensor& q = p.t[i];
      q.x = t[i].x;
      q.y = t[i].y;
      q.w = t[i].weight;
      q.xt = t[i].x_token, q.xh = t[i].x_head, q.yt = t[i].y_token, q.yh = t[i].y_head;
      q.heads = int(t[i].heads);
      const int64_t cap = std::max<int64_t>(1, std::min<int64_t>({32, kMaxPairs / (R / 2), T / 512}));
      q.tb = int(tokens_of_turn(q.heads, kThreads / p.L, cap));
      q.first = first;
      const int64_t turns = (T + q.tb - 1) / q.tb, share = std::max<int64_t>(1, resident * (q.heads + kSineHeads) / all);
      const int64_t each = (turns + share - 1) / share;
      q.blocks = int((turns + each - 1) / each);
      first += q.blocks;
      most = std::max(most, q.tb);
    }
    const size_t lds = size_t(most) * (R / 2) * sizeof(float2);
    hipLaunchKernelGGL(kernel, dim3(unsigned(first)), dim3(kThreads), lds, s, p);
  });
  return hipGetLastError();
}

NormBackwardPlan norm_backward_plan(int64_t T, int64_t D, int count, const int64_t* heads) {
  NormBackwardPlan plan{};
  int64_t all = 0;
  for (int i = 0; i < count; ++i) all += heads[i] + kSineHeads;
  for (int i = 0; i < count; ++i) {
    // four blocks per unit in all: 16384 tokens of 32 + 8 heads of 128, bf16, half layout, 113 us (before the second
    // launch's loads ran ahead: 108 now), interleaved 111; with three 108 and 120, with five 134 and 113
    const int64_t cap = std::max<int64_t>(1, 1024 * (heads[i] + kSineHeads) / all);
    const int64_t per = std::max<int64_t>(1, 2048 / (heads[i] * D));  // tokens a block takes at least
    plan.blocks[i] = int(std::max<int64_t>(1, std::min(cap, (T + per - 1) / per)));
    plan.offset[i] = plan.bytes;
    plan.bytes += plan.blocks[i] * D * 4;
  }
  return plan;
}

hipError_t launch_norm_rope_backward(int64_t T, int D, int R, int layout, int count, const qmv_norm_rope_grad* t, int dtype,
                                     int w_dtype, float eps, float offset, const int64_t* pos, const float* freqs,
                                     float amplitude, const NormBackwardPlan& plan, uint8_t* ws, hipStream_t s) {
  NormArgs p = common(T, D, R, count, w_dtype == QMV_F32, pos, freqs, amplitude, eps, offset);
  SumArgs sums{};
  sums.D = D;
  sums.w_f32 = p.w_f32;
  int J, first = 0, most = 1;
  bool any = false;
  shape_of(D, R, layout == QMV_ROPE_HALF, dtype, p.L, J);
  for (int i = 0; i < count; ++i) {
    NormTensor& q = p.t[i];
    q.x = t[i].x;
    q.dy = t[i].dy;
    q.y = t[i].dx;
    q.w = t[i].weight;
    q.xt = t[i].x_token, q.xh = t[i].x_head, q.gt = t[i].dy_token, q.gh = t[i].dy_head;
    q.yt = t[i].dx_token, q.yh = t[i].dx_head;
    q.heads = int(t[i].heads);
    q.first = first;
    q.blocks = plan.blocks[i];
    const int64_t turn_tokens = std::max<int64_t>(1, 8192 / (int64_t(q.heads) * D));
    q.tb = int(std::min<int64_t>({turn_tokens, std::max(1, kMaxPairs / (R / 2)), (T + q.blocks - 1) / q.blocks}));
    first += q.blocks;
    most = std::max(most, q.tb);
    if (t[i].dweight) {
      q.part = reinterpret_cast<float*>(ws + plan.offset[i]);
      sums.t[i] = {q.part, t[i].dweight, q.blocks};
      any = true;
    }
  }
  const size_t lds = std::max(size_t(most) * (R / 2) * sizeof(float2), size_t(4) * D * sizeof(float));
  dispatch(dtype, layout == QMV_ROPE_HALF, J, [&](auto e, auto h, auto j) {
    hipLaunchKernelGGL((norm_rope_backward_kernel<decltype(e)::value, decltype(h)::value, decltype(j)::value>),
                       dim3(unsigned(first)), dim3(kThreads), lds, s, p);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !any) return err;
  const dim3 grid(unsigned((D + 31) / 32), unsigned(count));
  if (dtype == QMV_F16) hipLaunchKernelGGL((norm_weight_kernel<1>), grid, dim3(1024), 0, s, sums);
  else if (dtype == QMV_BF16) hipLaunchKernelGGL((norm_weight_kernel<2>), grid, dim3(1024), 0, s, sums);
  else hipLaunchKernelGGL((norm_weight_kernel<0>), grid, dim3(1024), 0, s, sums);
  return hipGetLastError();
}

}  // namespace qmv
