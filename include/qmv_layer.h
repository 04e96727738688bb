/*
 * qmv_layer.h -- what a decoder layer over block-quantized weights needs around
 * the products of qmv.h when it takes many tokens at once: the gated
 * feed-forward products with their backward pass, and the rotary positions of
 * the q and k heads.  Same library (libqmv.so), same conventions as qmv.h:
 * packed layout, device pointers, caller-owned buffers, status codes and
 * qmv_last_error, streams, no allocation, no synchronization, graph capture.
 */
#ifndef QMV_LAYER_H_
#define QMV_LAYER_H_

#include "qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation of the gated products (qmv_gemm_glu). */
enum qmv_act {
  QMV_ACT_SILU = 1,      /* z / (1 + exp(-z)) */
  QMV_ACT_GELU_TANH = 2, /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
  QMV_ACT_GELU = 3       /* z/2 (1 + erf(z / sqrt 2)) */
};

/* Which values of a head form a rotary pair (qmv_rope). */
enum qmv_rope_layout {
  QMV_ROPE_HALF = 1,       /* (x[i], x[i + R/2]) */
  QMV_ROPE_INTERLEAVED = 2 /* (x[2i], x[2i + 1]) */
};

/* How qmv_rope_freqs stretches the frequencies for a longer context. */
enum qmv_rope_kind {
  QMV_ROPE_LINEAR = 1, /* every frequency divided by factor */
  QMV_ROPE_NTK = 2,    /* base multiplied by factor^(R / (R - 2)) */
  QMV_ROPE_PARTS = 3   /* by turns over the original context: slow pairs divided, fast ones kept */
};

/*
 * The gated feed-forward products of many tokens (aot-llm README, supported
 * architectures: SwiGLU / GeGLU), in one kernel:
 *   H[m][n] = act(g) * u,  g = sum_k X[m][k] W~g[n][k],  u = sum_k X[m][k] W~u[n][k]
 * for m < M, n < N.  W~ is the dequantized weight rounded once, to nearest
 * even, to x_dtype: the matrix cores take both operands in one 16-bit type
 * (QMV_F16: a weight past 65504 becomes an infinity; the packed scales themselves
 * are finite, and below 2^120 in QMV_I8_ROW).  Sums and the activation
 * are f32; every output is rounded once.
 *   fmt      any format; W_gate and W_up packed matrices of one shape
 *   X        [M][K] of x_dtype QMV_BF16 or QMV_F16, device, 16-byte aligned
 *   act      a qmv_act
 *   H        [M][N] of h_dtype == x_dtype, device, 16-byte aligned
 *   G, U     [M][N] of h_dtype, 16-byte aligned: receive g and u, which
 *            qmv_gemm_glu_backward needs; both or neither (NULL)
 * N >= 1, any M >= 1 (from single tokens to training batches); N, K <= 2^21,
 * M <= 2^30, M * N and M * K <= 2^34.  No output may overlap another buffer of
 * the call.  Within a row the result does not depend
 * on the other rows' values, and calls repeat bit for bit.
 * Errors: FORMAT, SHAPE, NULL, ALIGN, DTYPE, UNSUPPORTED (x_dtype f32 / Q8X, h_dtype other than
 * x_dtype, unknown act, buffers that overlap), OVERFLOW, DEVICE, LAUNCH.
 */
int qmv_gemm_glu(int fmt, int64_t N, int64_t K, int64_t M, const void* W_gate, const void* W_up, const void* X,
                 int x_dtype, int act, void* H, int h_dtype, void* G, void* U, void* stream);

/*
 * The backward pass of qmv_gemm_glu for a gradient dH of H:
 *   dG = dH * U * act'(G),  dU = dH * act(G)         (f32, each rounded once to dtype)
 *   dX[m][k] = sum_n dG[m][n] W~g[n][k] + dU[m][n] W~u[n][k]
 * with the rounded dG and dU and W~ as above (qmv_gemm_glu_backward_ex also takes them
 * unrounded); sums are f32, dX is rounded once.
 * The packed weights are constants (codes have no gradient); dG and dU are
 * what trainable matrices beside them (adapters) take their gradients from.
 *   G, U, dH, dG, dU   [M][N] of dtype (QMV_BF16 or QMV_F16), device, 16-byte aligned
 *   dX                 [M][K] of dtype, 16-byte aligned
 *   ws, ws_bytes       scratch memory, 16-byte aligned, of at least
 *                      qmv_gemm_glu_backward_bytes bytes (NULL if that is 0)
 * dG may be the buffer of G, U or dH, and dU that of another of them; outputs
 * otherwise overlap nothing.  Calls that overlap in time need a ws of their own.
 * Errors: as qmv_gemm_glu; SHAPE also for a ws_bytes that is too small.
 */
int qmv_gemm_glu_backward(int fmt, int64_t N, int64_t K, int64_t M, const void* W_gate, const void* W_up,
                          const void* G, const void* U, const void* dH, int dtype, int act, void* dG, void* dU,
                          void* dX, void* ws, size_t ws_bytes, void* stream);

/* Bytes of scratch memory that qmv_gemm_glu_backward needs for these sizes
 * (0: none).  Host only.  Errors: FORMAT, SHAPE, NULL, OVERFLOW. */
int qmv_gemm_glu_backward_bytes(int fmt, int64_t N, int64_t K, int64_t M, size_t* out_bytes);

/* What qmv_gemm_glu_backward_ex does otherwise than qmv_gemm_glu_backward. */
enum qmv_glu_flags {
  /* dX is the sum over dG and dU as they are before their rounding to dtype:
   * each enters the product as two 16-bit parts, the rounded value and what the
   * rounding left over (16 bits of it in bf16, 22 in f16, there down to multiples
   * of 2^-24).  dX is then off by its own rounding, where the sum over the rounded
   * dG and dU is off by about sqrt(2) of that, and by more where its terms cancel.
   * It takes twice the matrix operations.  Where dG or dU is past the type's
   * largest value, dX is infinite or NaN with it, and where W~ is infinite, dX of
   * that column is infinite or NaN. */
  QMV_GLU_UNROUNDED = 1
};

/* qmv_gemm_glu_backward with a set of qmv_glu_flags (0: the same call), and the
 * bytes of scratch memory that it needs with them.  dG and dU are the same with
 * any flags.  Errors: as the calls without _ex; UNSUPPORTED also for an unknown flag. */
int qmv_gemm_glu_backward_ex(int fmt, int64_t N, int64_t K, int64_t M, const void* W_gate, const void* W_up,
                             const void* G, const void* U, const void* dH, int dtype, int act, int flags, void* dG,
                             void* dU, void* dX, void* ws, size_t ws_bytes, void* stream);
int qmv_gemm_glu_backward_ex_bytes(int fmt, int64_t N, int64_t K, int64_t M, int flags, size_t* out_bytes);

/* One tensor of qmv_rope: T tokens of `heads` heads of D values; strides in
 * elements (values of a head are adjacent). */
#define QMV_ROPE_MAX 4
typedef struct qmv_rope_tensor {
  const void* x;
  void* y;          /* output; x itself with the same strides (in place), or no overlap with any x;
                       no overlap with another y, nor of its own values */
  int64_t heads;
  int64_t x_token, x_head;
  int64_t y_token, y_head;
} qmv_rope_tensor;

/*
 * Rotary positions (aot-llm README, Metal backend notes: RoPE on the q and k
 * projections; normal and NEOX pairings) of up to QMV_ROPE_MAX tensors in one
 * launch.  With t = pos[token] * freqs[i] for pair i < R/2 of every head,
 *   a' = amplitude * (a cos t - b sin t),  b' = amplitude * (b cos t + a sin t)
 * on the pairs (a, b) that `layout` names among the first R values of the
 * head; the other D - R values are copied.  inverse != 0 turns by -t: with the
 * same amplitude that is the gradient of the forward call.  The angle is
 * reduced in f64, so far positions (|pos| < 2^31) keep f32 accuracy; the
 * rotation is f32 and each output is rounded once to dtype.
 *   D >= 1, R even, 2 <= R <= D, R <= 4096; 1 <= count <= QMV_ROPE_MAX;
 *   T < 2^31, the tensors' heads together times D <= 2^28
 *   dtype     QMV_F32, QMV_F16 or QMV_BF16, of every x and y, aligned to its element
 *   pos       int64 [T], freqs f32 [R/2] (device)
 * Errors: SHAPE, NULL, ALIGN, DTYPE, UNSUPPORTED (Q8X, unknown layout, in place with other
 * strides, a y that is another tensor's x or y or holds values twice), OVERFLOW, DEVICE, LAUNCH.
 */
int qmv_rope(int64_t T, int64_t D, int64_t R, int layout, int count, const qmv_rope_tensor* tensors, int dtype,
             const int64_t* pos, const float* freqs, float amplitude, int inverse, void* stream);

/* A stretch of the rotary frequencies.  With f_i the frequency of pair i and
 * r_i = original * f_i / (2 pi) its turns over the original context,
 * QMV_ROPE_PARTS gives f_i (c + (1 - c) / factor), c = clamp((r_i - low) /
 * (high - low), 0, 1). */
typedef struct qmv_rope_scaling {
  int kind;        /* a qmv_rope_kind */
  double factor;   /* >= 1 */
  double original; /* PARTS: length of the original context, > 0 */
  double low;      /* PARTS: turns up to which a pair is divided by factor */
  double high;     /* PARTS: turns from which a pair is kept; > low */
} qmv_rope_scaling;

/*
 * freqs[i] = base^(-2i / R), i < R/2, stretched by `scaling` (NULL: not), as
 * f32 into host memory.  Host only; computed in f64 and rounded once.
 * Errors: SHAPE (R odd, < 2 or > 4096; NTK: R < 4), NULL, UNSUPPORTED (kind, a parameter that is
 * not finite or out of its range, or a frequency that f32 does not hold).
 */
int qmv_rope_freqs(int64_t R, double base, const qmv_rope_scaling* scaling, float* freqs);

#ifdef __cplusplus
}
#endif

#endif /* QMV_LAYER_H_ */
