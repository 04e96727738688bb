// C ABI of libqmv: argument validation, error reporting and dispatch.
//
// Unsupported or malformed requests are rejected on the host, before any
// launch, with a message naming the argument or the missing capability
// (aot-llm README: unsupported tensor types are rejected with a message
// naming the tensor; pytensor-ml issue 53, PR 18 acceptance rules: fail with
// the missing capability named, not at token 1).
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <utility>

#include "cache_internal.h"
#include "layer_internal.h"

namespace {

thread_local char g_last_error[256] = "";

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return status;
}

int ok() {
  g_last_error[0] = '\0';
  return QMV_OK;
}

const char* fmt_name(int fmt) {
  switch (fmt) {
    case QMV_Q8_0: return "Q8_0";
    case QMV_W4A16_G64: return "W4A16_G64";
    case QMV_Q4K: return "Q4K";
    case QMV_Q6K: return "Q6K";
    case QMV_Q4_0: return "Q4_0";
    case QMV_Q5_0: return "Q5_0";
    case QMV_Q5K: return "Q5K";
    case QMV_DENSE_BF16: return "DENSE_BF16";
    case QMV_I8_ROW: return "I8_ROW";
    default: return "?";
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Per-device architecture check, cached after the first query.
constexpr int kMaxDevices = 64;
std::atomic<int> g_dev_state[kMaxDevices];  // 0 unknown, 1 gfx950, -1 other

int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0)
    return fail(QMV_ERR_DEVICE, "hipGetDevice failed (no HIP device?)");
  if (dev < kMaxDevices) {
    const int st = g_dev_state[dev].load(std::memory_order_relaxed);
    if (st == 1) return QMV_OK;
    if (st == -1) return fail(QMV_ERR_DEVICE, "device %d is not gfx950", dev);
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
    return fail(QMV_ERR_DEVICE, "hipGetDeviceProperties(%d) failed", dev);
  const bool is950 = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDevices) g_dev_state[dev].store(is950 ? 1 : -1, std::memory_order_relaxed);
  if (!is950) return fail(QMV_ERR_DEVICE, "device %d is %s, the library is built for gfx950", dev,
                          prop.gcnArchName);
  return QMV_OK;
}

int check_fmt(int fmt) {
  if (qmv::block_of(fmt) == 0) return fail(QMV_ERR_FORMAT, "unknown format %d", fmt);
  return QMV_OK;
}

// N, K, batch sanity and size limits shared by all entry points.
int check_shape(int fmt, int64_t N, int64_t K, int64_t batch, const char* batch_name) {
  const int blk = qmv::block_of(fmt);
  if (N < 1) return fail(QMV_ERR_SHAPE, "N=%lld must be >= 1", (long long)N);
  if (K < 1) return fail(QMV_ERR_SHAPE, "K=%lld must be >= 1", (long long)K);
  if (K % blk) return fail(QMV_ERR_SHAPE, "K=%lld is not a multiple of the %s block (%d)",
                           (long long)K, fmt_name(fmt), blk);
  if (batch < 1) return fail(QMV_ERR_SHAPE, "%s=%lld must be >= 1", batch_name, (long long)batch);
  // kernels index rows and K with 32-bit ints and planes with 64-bit offsets
  const int64_t lim = int64_t(1) << 31;
  if (N >= lim || K >= lim) return fail(QMV_ERR_OVERFLOW, "N or K too large for 32-bit indexing");
  if (N > (int64_t(1) << 62) / K) return fail(QMV_ERR_OVERFLOW, "N*K overflows");
  return QMV_OK;
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

int launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(QMV_ERR_LAUNCH, "%s launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

int qmv_abi_version(int* layout_version) {
  if (layout_version) *layout_version = QMV_LAYOUT_VERSION;
  return QMV_ABI_VERSION;
}

const char* qmv_status_string(int status) {
  switch (status) {
    case QMV_OK: return "ok";
    case QMV_ERR_NULL: return "null pointer";
    case QMV_ERR_FORMAT: return "unknown format";
    case QMV_ERR_UNSUPPORTED: return "unsupported";
    case QMV_ERR_SHAPE: return "bad shape";
    case QMV_ERR_ALIGN: return "misaligned pointer";
    case QMV_ERR_DTYPE: return "bad dtype";
    case QMV_ERR_OVERFLOW: return "size overflow";
    case QMV_ERR_DEVICE: return "device error";
    case QMV_ERR_LAUNCH: return "launch failed";
    default: return "unknown status";
  }
}

const char* qmv_last_error(void) { return g_last_error; }

int qmv_packed_bytes(int fmt, int64_t N, int64_t K, int64_t batch, size_t* out_bytes) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if ((st = check_shape(fmt, N, K, batch, "batch"))) return st;
  if (!out_bytes) return fail(QMV_ERR_NULL, "out_bytes is NULL");
  const qmv::Planes p = qmv::planes_of(fmt, N, K);
  if (batch > INT64_MAX / p.total) return fail(QMV_ERR_OVERFLOW, "batch * packed bytes overflows");
  *out_bytes = static_cast<size_t>(batch * p.total);
  return ok();
}

int qmv_pack(int fmt, int64_t N, int64_t K, int64_t batch, const qmv_logical* src, void* dst,
             void* stream) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if ((st = check_shape(fmt, N, K, batch, "batch"))) return st;
  if (batch > 65535) return fail(QMV_ERR_OVERFLOW, "batch=%lld exceeds 65535", (long long)batch);
  if (!src) return fail(QMV_ERR_NULL, "src is NULL");
  if (!dst) return fail(QMV_ERR_NULL, "dst is NULL");
  if (!src->q) return fail(QMV_ERR_NULL, "src->q is NULL");
  const int naux = qmv::aux_count(fmt);
  for (int i = 0; i < naux; ++i)
    if (!src->aux[i]) return fail(QMV_ERR_NULL, "src->aux[%d] is NULL (%s needs %d)", i, fmt_name(fmt), naux);
  if (!aligned(dst, 16)) return fail(QMV_ERR_ALIGN, "dst is not 16-byte aligned");
  // f16 arrays (and the bf16 weights) 2-byte aligned, I8_ROW's f32 scales 4-byte
  const uintptr_t aux_align = fmt == QMV_I8_ROW ? 4 : 2;
  for (int i = 0; i < naux; ++i)
    if (!aligned(src->aux[i], aux_align))
      return fail(QMV_ERR_ALIGN, "src->aux[%d] is not %d-byte aligned", i, int(aux_align));
  if (fmt == QMV_DENSE_BF16 && !aligned(src->q, 2)) return fail(QMV_ERR_ALIGN, "src->q is not 2-byte aligned");
  const qmv::Planes p = qmv::planes_of(fmt, N, K);
  if (batch > INT64_MAX / p.total) return fail(QMV_ERR_OVERFLOW, "batch * packed bytes overflows");
  if ((N * K * (fmt == QMV_DENSE_BF16 ? 2 : 1) + 255) / 256 >= (int64_t(1) << 31))
    return fail(QMV_ERR_OVERFLOW, "matrix too large for one pack launch");
  if ((st = check_device())) return st;
  return launched(qmv::launch_pack(fmt, N, K, batch, *src, static_cast<uint8_t*>(dst), as_stream(stream)),
                  "pack");
}

static int check_matvec_args(int fmt, int64_t N, int64_t K, int64_t batch, const void* W, const void* x,
                             int x_dtype, const void* y, int y_dtype, const char* who) {
  int st;
  if ((st = check_shape(fmt, N, K, batch, "batch"))) {
    if (*who) {  // name the item
      char msg[sizeof(g_last_error)];
      std::snprintf(msg, sizeof(msg), "%s", g_last_error);
      fail(st, "%s%s", who, msg);
    }
    return st;
  }
  if (!W) return fail(QMV_ERR_NULL, "%sW is NULL", who);
  if (!x) return fail(QMV_ERR_NULL, "%sx is NULL", who);
  if (!y) return fail(QMV_ERR_NULL, "%sy is NULL", who);
  if (x_dtype != QMV_F32 && x_dtype != QMV_F16 && x_dtype != QMV_BF16 && x_dtype != QMV_Q8X)
    return fail(QMV_ERR_DTYPE, "x_dtype=%d is not a qmv_dtype", x_dtype);
  if (y_dtype != QMV_F32 && y_dtype != QMV_F16 && y_dtype != QMV_BF16 && y_dtype != QMV_Q8X)
    return fail(QMV_ERR_DTYPE, "y_dtype=%d is not a qmv_dtype", y_dtype);
  if (x_dtype == QMV_BF16 || (x_dtype == QMV_F16 && fmt != QMV_W4A16_G64) ||
      (x_dtype == QMV_Q8X && fmt == QMV_DENSE_BF16))
    return fail(QMV_ERR_UNSUPPORTED, "%s%s matvec takes x as f32%s", who, fmt_name(fmt),
                fmt == QMV_W4A16_G64 ? ", f16 or Q8X" : fmt == QMV_DENSE_BF16 ? "" : " or Q8X");
  if (y_dtype != QMV_F32) return fail(QMV_ERR_UNSUPPORTED, "matvec writes y as f32 only");
  if (!aligned(W, 16)) return fail(QMV_ERR_ALIGN, "%sW is not 16-byte aligned", who);
  if (!aligned(x, 16)) return fail(QMV_ERR_ALIGN, "%sx is not 16-byte aligned", who);
  if (!aligned(y, 4)) return fail(QMV_ERR_ALIGN, "%sy is not 4-byte aligned", who);
  const int64_t lim = int64_t(1) << 31;
  if (N * 16 >= lim) return fail(QMV_ERR_OVERFLOW, "N=%lld too large for the row grid", (long long)N);
  return QMV_OK;
}

int qmv_matvec(int fmt, int64_t N, int64_t K, int64_t batch, const void* W, const void* x,
               int x_dtype, void* y, int y_dtype, void* stream) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if ((st = check_matvec_args(fmt, N, K, batch, W, x, x_dtype, y, y_dtype, ""))) return st;
  if ((st = check_device())) return st;
  return launched(qmv::launch_matvec(fmt, N, K, batch, static_cast<const uint8_t*>(W), x, x_dtype,
                                     static_cast<float*>(y), as_stream(stream)),
                  "matvec");
}

int qmv_matvec_ex(int fmt, int64_t N, int64_t K, int64_t batch, const void* W, const void* x, int x_dtype,
                  void* y, int y_dtype, const qmv_epilogue* ep, void* stream) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if ((st = check_matvec_args(fmt, N, K, batch, W, x, x_dtype, y, y_dtype, ""))) return st;
  const float* bias = ep ? ep->bias : nullptr;
  const float* res = ep ? ep->residual : nullptr;
  if (bias && !aligned(bias, 4)) return fail(QMV_ERR_ALIGN, "ep->bias is not 4-byte aligned");
  if (res && !aligned(res, 4)) return fail(QMV_ERR_ALIGN, "ep->residual is not 4-byte aligned");
  if ((st = check_device())) return st;
  return launched(qmv::launch_matvec_epi(fmt, N, K, batch, static_cast<const uint8_t*>(W), nullptr, x, x_dtype,
                                         static_cast<float*>(y), bias, res, as_stream(stream)),
                  "matvec_ex");
}

int qmv_matvec_swiglu(int fmt, int64_t N, int64_t K, int64_t batch, const void* W_gate, const void* W_up,
                      const void* x, int x_dtype, void* h, int h_dtype, void* stream) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if (!W_gate) return fail(QMV_ERR_NULL, "W_gate is NULL");
  if (!W_up) return fail(QMV_ERR_NULL, "W_up is NULL");
  if ((st = check_matvec_args(fmt, N, K, batch, W_gate, x, x_dtype, h, h_dtype, ""))) return st;
  if (!aligned(W_up, 16)) return fail(QMV_ERR_ALIGN, "W_up is not 16-byte aligned");
  if ((st = check_device())) return st;
  return launched(qmv::launch_matvec_epi(fmt, N, K, batch, static_cast<const uint8_t*>(W_gate),
                                         static_cast<const uint8_t*>(W_up), x, x_dtype, static_cast<float*>(h),
                                         nullptr, nullptr, as_stream(stream)),
                  "matvec_swiglu");
}

int qmv_matvec_grouped(int fmt, int64_t K, int64_t batch, int count, const qmv_matvec_item* items,
                       int x_dtype, int y_dtype, void* stream) {
  int st;
  if (fmt != 0 && (st = check_fmt(fmt))) return st;
  if (count < 1 || count > 4096) return fail(QMV_ERR_SHAPE, "count=%d must be in [1, 4096]", count);
  if (!items) return fail(QMV_ERR_NULL, "items is NULL");
  char who[32];
  for (int i = 0; i < count; ++i) {
    std::snprintf(who, sizeof(who), "items[%d].", i);
    const int f = items[i].fmt ? items[i].fmt : fmt;
    if (f == 0) return fail(QMV_ERR_FORMAT, "%sfmt is 0 and the call's fmt is 0", who);
    if (qmv::block_of(f) == 0) return fail(QMV_ERR_FORMAT, "%sfmt=%d is not a qmv_format", who, f);
    if ((st = check_matvec_args(f, items[i].N, K, batch, items[i].W, items[i].x, x_dtype, items[i].y,
                                y_dtype, who)))
      return st;
  }
  if ((st = check_device())) return st;
  hipStream_t s = as_stream(stream);
  {
    hipError_t e = hipSuccess;
    if (batch == 1 ? qmv::launch_matvec_grouped_b1(fmt, K, count, items, x_dtype, s, &e)
                   : qmv::launch_matvec_grouped_mfma(fmt, K, batch, count, items, x_dtype, s, &e))
      return launched(e, "grouped matvec");
  }
  for (int i = 0; i < count; ++i) {
    const int f = items[i].fmt ? items[i].fmt : fmt;
    const hipError_t e = qmv::launch_matvec(f, items[i].N, K, batch, static_cast<const uint8_t*>(items[i].W),
                                            items[i].x, x_dtype, static_cast<float*>(items[i].y), s);
    if (e != hipSuccess) return launched(e, "grouped matvec");
  }
  return ok();
}

int qmv_gemm(int fmt, int64_t N, int64_t K, int64_t M, const void* W, const void* X, int x_dtype,
             void* Y, int y_dtype, void* stream) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if ((st = check_shape(fmt, N, K, M, "M"))) return st;
  if (!W) return fail(QMV_ERR_NULL, "W is NULL");
  if (!X) return fail(QMV_ERR_NULL, "X is NULL");
  if (!Y) return fail(QMV_ERR_NULL, "Y is NULL");
  if (x_dtype != QMV_F32 && x_dtype != QMV_F16 && x_dtype != QMV_BF16)
    return fail(QMV_ERR_DTYPE, "x_dtype=%d is not a qmv_dtype", x_dtype);
  if (y_dtype != QMV_F32 && y_dtype != QMV_F16 && y_dtype != QMV_BF16)
    return fail(QMV_ERR_DTYPE, "y_dtype=%d is not a qmv_dtype", y_dtype);
  if (fmt != QMV_W4A16_G64)
    return fail(QMV_ERR_UNSUPPORTED, "gemm supports W4A16_G64 only (got %s)", fmt_name(fmt));
  if (x_dtype != QMV_BF16 || y_dtype != QMV_BF16)
    return fail(QMV_ERR_UNSUPPORTED, "gemm takes X and writes Y as bf16");
  if (!aligned(W, 16)) return fail(QMV_ERR_ALIGN, "W is not 16-byte aligned");
  if (!aligned(X, 16)) return fail(QMV_ERR_ALIGN, "X is not 16-byte aligned");
  if (!aligned(Y, 4)) return fail(QMV_ERR_ALIGN, "Y is not 4-byte aligned");
  if (M >= (int64_t(1) << 31)) return fail(QMV_ERR_OVERFLOW, "M too large");
  if ((st = check_device())) return st;
  return launched(qmv::launch_gemm(fmt, N, K, M, static_cast<const uint8_t*>(W),
                                   static_cast<const uint16_t*>(X), static_cast<uint16_t*>(Y),
                                   as_stream(stream)),
                  "gemm");
}

int qmv_q8x_bytes(int64_t K, int64_t batch, size_t* out_bytes) {
  if (K < 32 || K % 32) return fail(QMV_ERR_SHAPE, "K=%lld must be a positive multiple of 32", (long long)K);
  if (batch < 1) return fail(QMV_ERR_SHAPE, "batch=%lld must be >= 1", (long long)batch);
  if (!out_bytes) return fail(QMV_ERR_NULL, "out_bytes is NULL");
  if (K >= (int64_t(1) << 31) || batch > (int64_t(1) << 40) / qmv::q8x_record_bytes(K))
    return fail(QMV_ERR_OVERFLOW, "batch * K too large");
  *out_bytes = static_cast<size_t>(batch * qmv::q8x_record_bytes(K));
  return ok();
}

int qmv_quantize_x(int64_t K, int64_t batch, const float* x, void* xq, void* stream) {
  int st;
  size_t bytes = 0;
  if ((st = qmv_q8x_bytes(K, batch, &bytes))) return st;
  if (!x) return fail(QMV_ERR_NULL, "x is NULL");
  if (!xq) return fail(QMV_ERR_NULL, "xq is NULL");
  if (!aligned(x, 16)) return fail(QMV_ERR_ALIGN, "x is not 16-byte aligned");
  if (!aligned(xq, 16)) return fail(QMV_ERR_ALIGN, "xq is not 16-byte aligned");
  if (batch * (K / 32) >= (int64_t(1) << 31) * 256)
    return fail(QMV_ERR_OVERFLOW, "too many blocks for one launch");
  if ((st = check_device())) return st;
  return launched(qmv::launch_quantize_x(K, batch, x, static_cast<uint8_t*>(xq), as_stream(stream)),
                  "quantize_x");
}

// 256 rows of N or K 16-bit values (and 256 packed rows) are reached by 31-bit byte offsets from
// their first; rows are counted in 31 bits with room for a tile, a launch's threads in 32.
static int check_glu_sizes(int64_t N, int64_t K, int64_t M) {
  if (N > (int64_t(1) << 21) || K > (int64_t(1) << 21)) return fail(QMV_ERR_OVERFLOW, "N or K is past 2^21");
  if (M > (int64_t(1) << 30) || M * N > (int64_t(1) << 34) || M * K > (int64_t(1) << 34))
    return fail(QMV_ERR_OVERFLOW, "M is past 2^30, or M * N or M * K past 2^34");
  return QMV_OK;
}

// Arguments that qmv_gemm_glu and its backward pass share.
static int check_glu(int fmt, int64_t N, int64_t K, int64_t M, const void* W_gate, const void* W_up, int dtype,
                     const char* dtype_name, int act) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if ((st = check_shape(fmt, N, K, M, "M"))) return st;
  if (!W_gate) return fail(QMV_ERR_NULL, "W_gate is NULL");
  if (!W_up) return fail(QMV_ERR_NULL, "W_up is NULL");
  if (dtype != QMV_F32 && dtype != QMV_F16 && dtype != QMV_BF16 && dtype != QMV_Q8X)
    return fail(QMV_ERR_DTYPE, "%s=%d is not a qmv_dtype", dtype_name, dtype);
  if (dtype != QMV_F16 && dtype != QMV_BF16)
    return fail(QMV_ERR_UNSUPPORTED, "the gated products take and write bf16 or f16");
  if (act < QMV_ACT_SILU || act > QMV_ACT_GELU) return fail(QMV_ERR_UNSUPPORTED, "act=%d is not a qmv_act", act);
  if (!aligned(W_gate, 16)) return fail(QMV_ERR_ALIGN, "W_gate is not 16-byte aligned");
  if (!aligned(W_up, 16)) return fail(QMV_ERR_ALIGN, "W_up is not 16-byte aligned");
  return check_glu_sizes(N, K, M);
}

static int check_buffer(const void* p, const char* name) {
  if (!p) return fail(QMV_ERR_NULL, "%s is NULL", name);
  if (!aligned(p, 16)) return fail(QMV_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return QMV_OK;
}

// Bytes [p, p + bytes) of a call's buffers.
struct Range {
  const void* p;
  int64_t bytes;
  const char* name;
};

// The workgroups of a launch read and write in no order: what one writes, none may read or write elsewhere.
static int check_apart(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (x < y + uintptr_t(b.bytes) && y < x + uintptr_t(a.bytes))
    return fail(QMV_ERR_UNSUPPORTED, "%s overlaps %s", a.name, b.name);
  return QMV_OK;
}

int qmv_gemm_glu(int fmt, int64_t N, int64_t K, int64_t M, const void* W_gate, const void* W_up, const void* X,
                 int x_dtype, int act, void* H, int h_dtype, void* G, void* U, void* stream) {
  int st;
  if ((st = check_glu(fmt, N, K, M, W_gate, W_up, x_dtype, "x_dtype", act))) return st;
  if (h_dtype != QMV_F32 && h_dtype != QMV_F16 && h_dtype != QMV_BF16 && h_dtype != QMV_Q8X)
    return fail(QMV_ERR_DTYPE, "h_dtype=%d is not a qmv_dtype", h_dtype);
  if (h_dtype != x_dtype) return fail(QMV_ERR_UNSUPPORTED, "h_dtype must be x_dtype");
  if ((st = check_buffer(X, "X"))) return st;
  if ((st = check_buffer(H, "H"))) return st;
  if ((G != nullptr) != (U != nullptr)) return fail(QMV_ERR_NULL, "%s is NULL and %s is not", G ? "U" : "G", G ? "G" : "U");
  if (G && ((st = check_buffer(G, "G")) || (st = check_buffer(U, "U")))) return st;
  if (H == X || G == X || U == X) return fail(QMV_ERR_UNSUPPORTED, "an output is the buffer of X");
  if (G && (G == H || U == H || G == U)) return fail(QMV_ERR_UNSUPPORTED, "two of H, G and U are one buffer");
  const Range rx{X, 2 * M * K, "X"}, out[] = {{H, 2 * M * N, "H"}, {G, 2 * M * N, "G"}, {U, 2 * M * N, "U"}};
  for (int i = 0; i < (G ? 3 : 1); ++i) {
    if ((st = check_apart(out[i], rx))) return st;
    for (int j = 0; j < i; ++j)
      if ((st = check_apart(out[i], out[j]))) return st;
  }
  if ((st = check_device())) return st;
  return launched(qmv::launch_glu_fwd(fmt, N, K, M, static_cast<const uint8_t*>(W_gate),
                                      static_cast<const uint8_t*>(W_up), static_cast<const uint16_t*>(X),
                                      x_dtype == QMV_F16, act, static_cast<uint16_t*>(H), static_cast<uint16_t*>(G),
                                      static_cast<uint16_t*>(U), as_stream(stream)),
                  "gemm_glu");
}

static size_t bytes_of(const qmv::GluBwdPlan& p) { return size_t(p.part_bytes + 2 * p.copy_bytes + 2 * p.low_bytes); }

static int check_glu_flags(int flags) {
  if (flags & ~QMV_GLU_UNROUNDED) return fail(QMV_ERR_UNSUPPORTED, "flags=%d holds an unknown flag", flags);
  return QMV_OK;
}

int qmv_gemm_glu_backward_bytes(int fmt, int64_t N, int64_t K, int64_t M, size_t* out_bytes) {
  return qmv_gemm_glu_backward_ex_bytes(fmt, N, K, M, 0, out_bytes);
}

int qmv_gemm_glu_backward_ex_bytes(int fmt, int64_t N, int64_t K, int64_t M, int flags, size_t* out_bytes) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if ((st = check_shape(fmt, N, K, M, "M"))) return st;
  if (!out_bytes) return fail(QMV_ERR_NULL, "out_bytes is NULL");
  if ((st = check_glu_flags(flags))) return st;
  if ((st = check_glu_sizes(N, K, M))) return st;
  *out_bytes = bytes_of(qmv::glu_backward_plan(N, K, M, flags & QMV_GLU_UNROUNDED));
  return ok();
}

int qmv_gemm_glu_backward(int fmt, int64_t N, int64_t K, int64_t M, const void* W_gate, const void* W_up,
                          const void* G, const void* U, const void* dH, int dtype, int act, void* dG, void* dU,
                          void* dX, void* ws, size_t ws_bytes, void* stream) {
  return qmv_gemm_glu_backward_ex(fmt, N, K, M, W_gate, W_up, G, U, dH, dtype, act, 0, dG, dU, dX, ws, ws_bytes, stream);
}

int qmv_gemm_glu_backward_ex(int fmt, int64_t N, int64_t K, int64_t M, const void* W_gate, const void* W_up,
                             const void* G, const void* U, const void* dH, int dtype, int act, int flags, void* dG,
                             void* dU, void* dX, void* ws, size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_glu(fmt, N, K, M, W_gate, W_up, dtype, "dtype", act))) return st;
  if ((st = check_glu_flags(flags))) return st;
  const void* bufs[] = {G, U, dH, dG, dU, dX};
  const char* names[] = {"G", "U", "dH", "dG", "dU", "dX"};
  for (int i = 0; i < 6; ++i)
    if ((st = check_buffer(bufs[i], names[i]))) return st;
  if (dG == dU) return fail(QMV_ERR_UNSUPPORTED, "dG and dU are the same buffer");
  for (int i = 0; i < 5; ++i)
    if (dX == bufs[i]) return fail(QMV_ERR_UNSUPPORTED, "dX is the buffer of %s", names[i]);
  const qmv::GluBwdPlan plan = qmv::glu_backward_plan(N, K, M, flags & QMV_GLU_UNROUNDED);
  const size_t need = bytes_of(plan);
  if (need) {
    if ((st = check_buffer(ws, "ws"))) return st;
    if (ws_bytes < need)
      return fail(QMV_ERR_SHAPE, "ws_bytes=%llu, the call needs %llu", (unsigned long long)ws_bytes,
                  (unsigned long long)need);
  }
  Range r[7];
  for (int i = 0; i < 6; ++i) r[i] = Range{bufs[i], 2 * M * (i == 5 ? K : N), names[i]};
  r[6] = Range{ws, int64_t(need), "ws"};
  for (int i = 3; i < (need ? 7 : 6); ++i)  // dG and dU may be G, U or dH, as a whole
    for (int j = 0; j < i; ++j)
      if (!(i < 5 && j < 3 && r[i].p == r[j].p) && (st = check_apart(r[i], r[j]))) return st;
  if ((st = check_device())) return st;
  return launched(qmv::launch_glu_bwd(fmt, N, K, M, static_cast<const uint8_t*>(W_gate),
                                      static_cast<const uint8_t*>(W_up), static_cast<const uint16_t*>(G),
                                      static_cast<const uint16_t*>(U), static_cast<const uint16_t*>(dH),
                                      dtype == QMV_F16, act, plan, static_cast<uint16_t*>(dG),
                                      static_cast<uint16_t*>(dU), static_cast<uint16_t*>(dX), static_cast<uint8_t*>(ws),
                                      as_stream(stream)),
                  "gemm_glu_backward");
}

int qmv_rope(int64_t T, int64_t D, int64_t R, int layout, int count, const qmv_rope_tensor* tensors, int dtype,
             const int64_t* pos, const float* freqs, float amplitude, int inverse, void* stream) {
  int st;
  if (T < 1) return fail(QMV_ERR_SHAPE, "T=%lld must be >= 1", (long long)T);
  if (D < 1) return fail(QMV_ERR_SHAPE, "D=%lld must be >= 1", (long long)D);
  if (R < 2 || R % 2 || R > D || R > 4096)
    return fail(QMV_ERR_SHAPE, "R=%lld must be even, in [2, min(D, 4096)] (D=%lld)", (long long)R, (long long)D);
  if (layout != QMV_ROPE_HALF && layout != QMV_ROPE_INTERLEAVED)
    return fail(QMV_ERR_UNSUPPORTED, "layout=%d is not a qmv_rope_layout", layout);
  if (count < 1 || count > QMV_ROPE_MAX)
    return fail(QMV_ERR_SHAPE, "count=%d must be in [1, %d]", count, QMV_ROPE_MAX);
  if (!tensors) return fail(QMV_ERR_NULL, "tensors is NULL");
  if (!pos) return fail(QMV_ERR_NULL, "pos is NULL");
  if (!freqs) return fail(QMV_ERR_NULL, "freqs is NULL");
  if (dtype != QMV_F32 && dtype != QMV_F16 && dtype != QMV_BF16 && dtype != QMV_Q8X)
    return fail(QMV_ERR_DTYPE, "dtype=%d is not a qmv_dtype", dtype);
  if (dtype == QMV_Q8X) return fail(QMV_ERR_UNSUPPORTED, "rope takes f32, f16 or bf16");
  if (!aligned(pos, 8)) return fail(QMV_ERR_ALIGN, "pos is not 8-byte aligned");
  if (!aligned(freqs, 4)) return fail(QMV_ERR_ALIGN, "freqs is not 4-byte aligned");
  const int64_t lim = int64_t(1) << 31;
  int64_t heads = 0;
  for (int i = 0; i < count; ++i) {
    const qmv_rope_tensor& t = tensors[i];
    if (t.heads < 1) return fail(QMV_ERR_SHAPE, "tensors[%d].heads=%lld must be >= 1", i, (long long)t.heads);
    if (!t.x) return fail(QMV_ERR_NULL, "tensors[%d].x is NULL", i);
    if (!t.y) return fail(QMV_ERR_NULL, "tensors[%d].y is NULL", i);
    if (!aligned(t.x, dtype == QMV_F32 ? 4 : 2)) return fail(QMV_ERR_ALIGN, "tensors[%d].x is not aligned to its element", i);
    if (!aligned(t.y, dtype == QMV_F32 ? 4 : 2)) return fail(QMV_ERR_ALIGN, "tensors[%d].y is not aligned to its element", i);
    if (t.x == t.y && (t.x_token != t.y_token || t.x_head != t.y_head))
      return fail(QMV_ERR_UNSUPPORTED, "tensors[%d] is in place with other strides", i);
    if (t.heads >= lim) return fail(QMV_ERR_OVERFLOW, "tensors[%d].heads too large", i);
    heads += t.heads;
  }
  // one launch turns all tensors, in no order
  for (int i = 0; i < count; ++i)
    for (int j = 0; j < count; ++j) {
      if (i < j && tensors[i].y == tensors[j].y)
        return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].y and tensors[%d].y are one buffer", i, j);
      if (i != j && tensors[i].y == tensors[j].x)
        return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].y is the buffer of tensors[%d].x", i, j);
    }
  // a block of tokens is indexed with 32-bit ints, the grid counts tokens
  if (D > (lim >> 3) || heads > (lim >> 3) / D || T >= lim)
    return fail(QMV_ERR_OVERFLOW, "T is past 2^31 or heads * D past 2^28");
  // tokens and heads of an output: the larger stride passes what the smaller one reaches
  for (int i = 0; i < count; ++i) {
    const qmv_rope_tensor& t = tensors[i];
    struct Axis {
      int64_t n, st;
    } in{t.heads, std::llabs(t.y_head)}, out{T, std::llabs(t.y_token)};
    if (in.n > 1 && out.n > 1 && in.st > out.st) std::swap(in, out);
    if (in.n > 1 && in.st < D) return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].y holds some values more than once", i);
    const int64_t reach = in.n > 1 ? (in.n - 1) * in.st + D : D;
    if (out.n > 1 && out.st < reach) return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].y holds some values more than once", i);
  }
  if ((st = check_device())) return st;
  return launched(qmv::launch_rope(T, int(D), int(R), layout, count, tensors, dtype, pos, freqs, amplitude, inverse,
                                   as_stream(stream)),
                  "rope");
}

// Heads of T tokens that lie at strides: an output's own values must not meet.
static bool meets_itself(int64_t T, int64_t D, int64_t heads, int64_t token, int64_t head) {
  struct Axis {
    int64_t n, st;
  } in{heads, std::llabs(head)}, out{T, std::llabs(token)};
  if (in.n > 1 && out.n > 1 && in.st > out.st) std::swap(in, out);
  const int64_t reach = in.n > 1 ? (in.n - 1) * in.st + D : D;
  return (in.n > 1 && in.st < D) || (out.n > 1 && out.st < reach);
}

static bool is_dtype(int d) { return d == QMV_F32 || d == QMV_F16 || d == QMV_BF16 || d == QMV_Q8X; }
static uintptr_t element(int dtype) { return dtype == QMV_F32 ? 4 : 2; }

// Arguments that qmv_norm_rope and its backward pass share.
static int check_norm_rope(int64_t T, int64_t D, int64_t R, int layout, int count, const void* tensors, int dtype,
                           int w_dtype, float eps, float w_offset, const int64_t* pos, const float* freqs) {
  if (T < 1) return fail(QMV_ERR_SHAPE, "T=%lld must be >= 1", (long long)T);
  if (D < 1 || D > 1024) return fail(QMV_ERR_SHAPE, "D=%lld must be in [1, 1024]", (long long)D);
  if (R < 2 || R % 2 || R > D)
    return fail(QMV_ERR_SHAPE, "R=%lld must be even, in [2, D] (D=%lld)", (long long)R, (long long)D);
  if (layout != QMV_ROPE_HALF && layout != QMV_ROPE_INTERLEAVED)
    return fail(QMV_ERR_UNSUPPORTED, "layout=%d is not a qmv_rope_layout", layout);
  if (count < 1 || count > QMV_ROPE_MAX)
    return fail(QMV_ERR_SHAPE, "count=%d must be in [1, %d]", count, QMV_ROPE_MAX);
  if (!tensors) return fail(QMV_ERR_NULL, "tensors is NULL");
  if (!pos) return fail(QMV_ERR_NULL, "pos is NULL");
  if (!freqs) return fail(QMV_ERR_NULL, "freqs is NULL");
  if (!is_dtype(dtype)) return fail(QMV_ERR_DTYPE, "dtype=%d is not a qmv_dtype", dtype);
  if (dtype == QMV_Q8X) return fail(QMV_ERR_UNSUPPORTED, "norm_rope takes f32, f16 or bf16");
  if (w_dtype != QMV_F32 && w_dtype != dtype)
    return fail(QMV_ERR_DTYPE, "w_dtype=%d must be QMV_F32 or dtype", w_dtype);
  if (!(std::isfinite(eps) && eps >= 0)) return fail(QMV_ERR_UNSUPPORTED, "eps must be finite and >= 0");
  if (!std::isfinite(w_offset)) return fail(QMV_ERR_UNSUPPORTED, "w_offset must be finite");
  if (!aligned(pos, 8)) return fail(QMV_ERR_ALIGN, "pos is not 8-byte aligned");
  if (!aligned(freqs, 4)) return fail(QMV_ERR_ALIGN, "freqs is not 4-byte aligned");
  if (T >= (int64_t(1) << 31)) return fail(QMV_ERR_OVERFLOW, "T is past 2^31");
  return QMV_OK;
}

// heads of each tensor: a block of tokens is indexed with 32-bit ints
static int check_heads(int64_t D, int count, const int64_t* heads) {
  int64_t all = 0;
  for (int i = 0; i < count; ++i) {
    if (heads[i] < 1) return fail(QMV_ERR_SHAPE, "tensors[%d].heads=%lld must be >= 1", i, (long long)heads[i]);
    if (heads[i] > (int64_t(1) << 28)) return fail(QMV_ERR_OVERFLOW, "tensors[%d].heads too large", i);
    all += heads[i];
  }
  if (all > (int64_t(1) << 28) / D) return fail(QMV_ERR_OVERFLOW, "heads * D past 2^28");
  return QMV_OK;
}

static int check_place(const void* p, uintptr_t align, int i, const char* name) {
  if (!p) return fail(QMV_ERR_NULL, "tensors[%d].%s is NULL", i, name);
  if (!aligned(p, align)) return fail(QMV_ERR_ALIGN, "tensors[%d].%s is not aligned to its element", i, name);
  return QMV_OK;
}

int qmv_norm_rope(int64_t T, int64_t D, int64_t R, int layout, int count, const qmv_norm_rope_tensor* tensors, int dtype,
                  int w_dtype, float eps, float w_offset, const int64_t* pos, const float* freqs, float amplitude,
                  void* stream) {
  int st;
  if ((st = check_norm_rope(T, D, R, layout, count, tensors, dtype, w_dtype, eps, w_offset, pos, freqs))) return st;
  int64_t heads[QMV_ROPE_MAX];
  for (int i = 0; i < count; ++i) heads[i] = tensors[i].heads;
  if ((st = check_heads(D, count, heads))) return st;
  for (int i = 0; i < count; ++i) {
    const qmv_norm_rope_tensor& t = tensors[i];
    if ((st = check_place(t.x, element(dtype), i, "x"))) return st;
    if ((st = check_place(t.y, element(dtype), i, "y"))) return st;
    if (t.weight && (st = check_place(t.weight, element(w_dtype), i, "weight"))) return st;
    if (t.x == t.y && (t.x_token != t.y_token || t.x_head != t.y_head))
      return fail(QMV_ERR_UNSUPPORTED, "tensors[%d] is in place with other strides", i);
    if (meets_itself(T, D, t.heads, t.y_token, t.y_head))
      return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].y holds some values more than once", i);
  }
  for (int i = 0; i < count; ++i)  // one launch works on all tensors, in no order
    for (int j = 0; j < count; ++j) {
      if (i < j && tensors[i].y == tensors[j].y)
        return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].y and tensors[%d].y are one buffer", i, j);
      if (i != j && tensors[i].y == tensors[j].x)
        return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].y is the buffer of tensors[%d].x", i, j);
      if (tensors[i].y == tensors[j].weight)
        return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].y is the buffer of tensors[%d].weight", i, j);
    }
  if ((st = check_device())) return st;
  return launched(qmv::launch_norm_rope(T, int(D), int(R), layout, count, tensors, dtype, w_dtype, eps, w_offset, pos, freqs,
                                        amplitude, as_stream(stream)),
                  "norm_rope");
}

int qmv_norm_rope_backward_bytes(int64_t T, int64_t D, int count, const int64_t* heads, size_t* out_bytes) {
  int st;
  if (T < 1) return fail(QMV_ERR_SHAPE, "T=%lld must be >= 1", (long long)T);
  if (D < 1 || D > 1024) return fail(QMV_ERR_SHAPE, "D=%lld must be in [1, 1024]", (long long)D);
  if (count < 1 || count > QMV_ROPE_MAX)
    return fail(QMV_ERR_SHAPE, "count=%d must be in [1, %d]", count, QMV_ROPE_MAX);
  if (!heads) return fail(QMV_ERR_NULL, "heads is NULL");
  if (!out_bytes) return fail(QMV_ERR_NULL, "out_bytes is NULL");
  if (T >= (int64_t(1) << 31)) return fail(QMV_ERR_OVERFLOW, "T is past 2^31");
  if ((st = check_heads(D, count, heads))) return st;
  *out_bytes = size_t(qmv::norm_backward_plan(T, D, count, heads).bytes);
  return ok();
}

int qmv_norm_rope_backward(int64_t T, int64_t D, int64_t R, int layout, int count, const qmv_norm_rope_grad* tensors,
                           int dtype, int w_dtype, float eps, float w_offset, const int64_t* pos, const float* freqs,
                           float amplitude, void* ws, size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_norm_rope(T, D, R, layout, count, tensors, dtype, w_dtype, eps, w_offset, pos, freqs))) return st;
  int64_t heads[QMV_ROPE_MAX];
  for (int i = 0; i < count; ++i) heads[i] = tensors[i].heads;
  if ((st = check_heads(D, count, heads))) return st;
  bool sums = false;
  for (int i = 0; i < count; ++i) {
    const qmv_norm_rope_grad& t = tensors[i];
    if ((st = check_place(t.x, element(dtype), i, "x"))) return st;
    if ((st = check_place(t.dy, element(dtype), i, "dy"))) return st;
    if ((st = check_place(t.dx, element(dtype), i, "dx"))) return st;
    if (t.weight && (st = check_place(t.weight, element(w_dtype), i, "weight"))) return st;
    if (t.dweight) {
      if (!t.weight) return fail(QMV_ERR_NULL, "tensors[%d].dweight is given without weight", i);
      if ((st = check_place(t.dweight, element(w_dtype), i, "dweight"))) return st;
      sums = true;
    }
    if ((t.dx == t.x && (t.dx_token != t.x_token || t.dx_head != t.x_head)) ||
        (t.dx == t.dy && (t.dx_token != t.dy_token || t.dx_head != t.dy_head)))
      return fail(QMV_ERR_UNSUPPORTED, "tensors[%d] is in place with other strides", i);
    if (meets_itself(T, D, t.heads, t.dx_token, t.dx_head))
      return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].dx holds some values more than once", i);
  }
  const qmv::NormBackwardPlan plan = qmv::norm_backward_plan(T, D, count, heads);
  if (sums) {
    if (!ws) return fail(QMV_ERR_NULL, "ws is NULL");
    if (!aligned(ws, 16)) return fail(QMV_ERR_ALIGN, "ws is not 16-byte aligned");
    if (ws_bytes < size_t(plan.bytes))
      return fail(QMV_ERR_SHAPE, "ws_bytes=%llu, the call needs %lld", (unsigned long long)ws_bytes, (long long)plan.bytes);
  }
  const int64_t wb = D * int64_t(element(w_dtype));
  for (int i = 0; i < count; ++i)
    for (int j = 0; j < count; ++j) {
      const qmv_norm_rope_grad &a = tensors[i], &b = tensors[j];
      if (i < j && a.dx == b.dx) return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].dx and tensors[%d].dx are one buffer", i, j);
      if (i != j && (a.dx == b.x || a.dx == b.dy))
        return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].dx is the buffer of tensors[%d].%s", i, j, a.dx == b.x ? "x" : "dy");
      if (a.dx == b.weight) return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].dx is the buffer of tensors[%d].weight", i, j);
      if (!a.dweight) continue;
      // the launch that writes a dweight runs after the one that reads the inputs; the weights may
      // serve the next call, so what it writes is apart from all but its own
      const Range r{a.dweight, wb, "dweight"};
      if (b.weight && (st = check_apart(r, Range{b.weight, wb, "weight"}))) return st;
      if (i < j && b.dweight && (st = check_apart(r, Range{b.dweight, wb, "another dweight"}))) return st;
      if (a.dweight == b.x || a.dweight == b.dy || a.dweight == b.dx)
        return fail(QMV_ERR_UNSUPPORTED, "tensors[%d].dweight is the buffer of tensors[%d].x, dy or dx", i, j);
      const Range w{ws, plan.bytes, "ws"};
      if ((st = check_apart(w, r))) return st;
      if (b.weight && (st = check_apart(w, Range{b.weight, wb, "weight"}))) return st;
      if (b.x == ws || b.dy == ws || b.dx == ws) return fail(QMV_ERR_UNSUPPORTED, "ws is the buffer of tensors[%d].x, dy or dx", j);
    }
  if ((st = check_device())) return st;
  return launched(qmv::launch_norm_rope_backward(T, int(D), int(R), layout, count, tensors, dtype, w_dtype, eps, w_offset, pos,
                                                 freqs, amplitude, plan, static_cast<uint8_t*>(ws), as_stream(stream)),
                  "norm_rope_backward");
}

// ------------------------------------------------------ key / value cache

static int check_cache(const qmv_kv_cache* c, bool with_data) {
  if (!c) return fail(QMV_ERR_NULL, "cache is NULL");
  if (c->fmt != QMV_Q8_0 && c->fmt != QMV_Q4_0)
    return fail(QMV_ERR_FORMAT, "cache->fmt=%d must be QMV_Q8_0 or QMV_Q4_0", int(c->fmt));
  if (c->page < 16 || c->page % 16 || c->page > 1024)
    return fail(QMV_ERR_SHAPE, "cache->page=%d must be a multiple of 16, at most 1024", int(c->page));
  if (c->D < 32 || c->D % 32 || c->D > 256)
    return fail(QMV_ERR_SHAPE, "cache->D=%lld must be a multiple of 32, at most 256", (long long)c->D);
  if (c->heads < 1) return fail(QMV_ERR_SHAPE, "cache->heads=%lld must be >= 1", (long long)c->heads);
  if (c->pages < 1) return fail(QMV_ERR_SHAPE, "cache->pages=%lld must be >= 1", (long long)c->pages);
  if (c->heads > 65535) return fail(QMV_ERR_OVERFLOW, "cache->heads is past 65535");
  if (c->pages > 0x7FFFFFFF) return fail(QMV_ERR_OVERFLOW, "cache->pages is past 2^31 - 1");
  if (with_data) {
    if (!c->data) return fail(QMV_ERR_NULL, "cache->data is NULL");
    if (!aligned(c->data, 16)) return fail(QMV_ERR_ALIGN, "cache->data is not 16-byte aligned");
  }
  return QMV_OK;
}

static int64_t cache_bytes(const qmv_kv_cache& c) {  // below 2^31 * 2^16 * 2^20 at most
  return c.pages * c.heads * (c.page / 16) * qmv::kv_set_bytes(c.fmt, c.D);
}

int qmv_kv_cache_bytes(const qmv_kv_cache* cache, size_t* out_bytes) {
  int st;
  if ((st = check_cache(cache, false))) return st;
  if (!out_bytes) return fail(QMV_ERR_NULL, "out_bytes is NULL");
  if (cache->pages > (int64_t(1) << 50) / (cache->heads << 20)) return fail(QMV_ERR_OVERFLOW, "the cache is past 2^50 bytes");
  *out_bytes = size_t(cache_bytes(*cache));
  return ok();
}

static int check_batch(const qmv_kv_cache* c, const qmv_kv_batch* b, bool with_pointers) {
  if (!b) return fail(QMV_ERR_NULL, "batch is NULL");
  if (b->T < 1) return fail(QMV_ERR_SHAPE, "batch->T=%lld must be >= 1", (long long)b->T);
  if (b->B < 1) return fail(QMV_ERR_SHAPE, "batch->B=%lld must be >= 1", (long long)b->B);
  if (b->columns < 1) return fail(QMV_ERR_SHAPE, "batch->columns=%lld must be >= 1", (long long)b->columns);
  if (b->T >= (int64_t(1) << 31)) return fail(QMV_ERR_OVERFLOW, "batch->T is past 2^31");
  // a launch has a workgroup for each sequence and head, and counts threads in 32 bits
  if (b->B > (int64_t(1) << 23) / c->heads) return fail(QMV_ERR_OVERFLOW, "batch->B * heads is past 2^23");
  if (b->columns > (int64_t(1) << 30) / c->page) return fail(QMV_ERR_OVERFLOW, "batch->columns * page is past 2^30");
  if (!with_pointers) return QMV_OK;
  if (b->B > 1 && b->stride < b->columns)
    return fail(QMV_ERR_SHAPE, "batch->stride=%lld is below columns=%lld", (long long)b->stride, (long long)b->columns);
  if (!b->q_start) return fail(QMV_ERR_NULL, "batch->q_start is NULL");
  if (!b->kv_len) return fail(QMV_ERR_NULL, "batch->kv_len is NULL");
  if (!b->table) return fail(QMV_ERR_NULL, "batch->table is NULL");
  if (!aligned(b->q_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->table, 4))
    return fail(QMV_ERR_ALIGN, "batch->q_start, kv_len or table is not 4-byte aligned");
  return QMV_OK;
}

// From the first to the last byte of strided heads (what lies between them may be another tensor's).
static Range reach(const void* p, int64_t T, int64_t heads, int64_t D, int64_t token, int64_t head, int dtype,
                   const char* name) {
  typedef __int128 Wide;
  const Wide t = Wide(T - 1) * token, h = Wide(heads - 1) * head, most = Wide(1) << 46;
  const Wide lo = std::max<Wide>(-most, (t < 0 ? t : 0) + (h < 0 ? h : 0));
  const Wide hi = std::min<Wide>(most, (t > 0 ? t : 0) + (h > 0 ? h : 0) + D);
  const int64_t e = int64_t(element(dtype));
  const uintptr_t from = reinterpret_cast<uintptr_t>(p) + uintptr_t(int64_t(lo) * e);
  return Range{reinterpret_cast<const void*>(from), int64_t(hi - lo) * e, name};
}

static bool in_cache(const qmv_kv_cache& c, const Range& r) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(r.p), d = reinterpret_cast<uintptr_t>(c.data);
  return x < d + uintptr_t(cache_bytes(c)) && d < x + uintptr_t(r.bytes);
}

static int check_kv_dtype(int dtype) {
  if (!is_dtype(dtype)) return fail(QMV_ERR_DTYPE, "dtype=%d is not a qmv_dtype", dtype);
  if (dtype == QMV_Q8X) return fail(QMV_ERR_UNSUPPORTED, "the cache takes and gives f32, f16 or bf16");
  return QMV_OK;
}

static int check_kv(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const void* k, int64_t k_token, int64_t k_head,
                    const void* v, int64_t v_token, int64_t v_head, int dtype) {
  int st;
  size_t bytes;
  if ((st = check_cache(cache, true))) return st;
  if ((st = qmv_kv_cache_bytes(cache, &bytes))) return st;
  if ((st = check_batch(cache, batch, true))) return st;
  if ((st = check_kv_dtype(dtype))) return st;
  const void* p[] = {k, v};
  const int64_t token[] = {k_token, v_token}, head[] = {k_head, v_head};
  const char* names[] = {"k", "v"};
  for (int i = 0; i < 2; ++i) {
    if (!p[i]) continue;
    if (!aligned(p[i], element(dtype))) return fail(QMV_ERR_ALIGN, "%s is not aligned to its element", names[i]);
    if (in_cache(*cache, reach(p[i], batch->T, cache->heads, cache->D, token[i], head[i], dtype, names[i])))
      return fail(QMV_ERR_UNSUPPORTED, "%s lies in the cache", names[i]);
  }
  return QMV_OK;
}

int qmv_kv_write(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const void* k, int64_t k_token, int64_t k_head,
                 const void* v, int64_t v_token, int64_t v_head, int dtype, void* stream) {
  int st;
  if ((st = check_kv(cache, batch, k, k_token, k_head, v, v_token, v_head, dtype))) return st;
  if (!k) return fail(QMV_ERR_NULL, "k is NULL");
  if (!v) return fail(QMV_ERR_NULL, "v is NULL");
  if ((st = check_device())) return st;
  return launched(qmv::launch_kv_write(*cache, *batch, k, k_token, k_head, v, v_token, v_head, dtype, as_stream(stream)),
                  "kv_write");
}

int qmv_kv_read(const qmv_kv_cache* cache, const qmv_kv_batch* batch, void* k, int64_t k_token, int64_t k_head, void* v,
                int64_t v_token, int64_t v_head, int dtype, void* stream) {
  int st;
  if ((st = check_kv(cache, batch, k, k_token, k_head, v, v_token, v_head, dtype))) return st;
  if (!k && !v) return fail(QMV_ERR_NULL, "k and v are NULL");
  if (k && meets_itself(batch->T, cache->D, cache->heads, k_token, k_head))
    return fail(QMV_ERR_UNSUPPORTED, "k holds some values more than once");
  if (v && meets_itself(batch->T, cache->D, cache->heads, v_token, v_head))
    return fail(QMV_ERR_UNSUPPORTED, "v holds some values more than once");
  if (k == v) return fail(QMV_ERR_UNSUPPORTED, "k and v are one buffer");
  if ((st = check_device())) return st;
  return launched(qmv::launch_kv_read(*cache, *batch, k, k_token, k_head, v, v_token, v_head, dtype, as_stream(stream)),
                  "kv_read");
}

static int check_attention_sizes(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const qmv_kv_attention_args* a,
                                 bool call) {
  int st;
  size_t bytes;
  if ((st = check_cache(cache, call))) return st;
  if ((st = qmv_kv_cache_bytes(cache, &bytes))) return st;
  if ((st = check_batch(cache, batch, call))) return st;
  if (!a) return fail(QMV_ERR_NULL, "args is NULL");
  if (a->q_heads < 1 || a->q_heads % cache->heads)
    return fail(QMV_ERR_SHAPE, "args->q_heads=%lld must be a multiple of the cache's heads (%lld)", (long long)a->q_heads,
                (long long)cache->heads);
  if ((st = check_kv_dtype(a->dtype))) return st;
  if (a->window < 0) return fail(QMV_ERR_SHAPE, "args->window=%lld must be >= 0", (long long)a->window);
  if (a->prefix < 0) return fail(QMV_ERR_SHAPE, "args->prefix=%lld must be >= 0", (long long)a->prefix);
  if (a->max_q < 1) return fail(QMV_ERR_SHAPE, "args->max_q=%lld must be >= 1", (long long)a->max_q);
  if (a->max_kv < 1) return fail(QMV_ERR_SHAPE, "args->max_kv=%lld must be >= 1", (long long)a->max_kv);
  // the rows of a k / v head are counted in 32 bits, with room for a tile
  if (a->q_heads > (int64_t(1) << 20) || a->q_heads / cache->heads > (int64_t(1) << 30) / batch->T)
    return fail(QMV_ERR_OVERFLOW, "args->q_heads is past 2^20, or T * q_heads / heads past 2^30");
  return QMV_OK;
}

int qmv_kv_attention_bytes(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const qmv_kv_attention_args* args,
                           size_t* out_bytes) {
  int st;
  if ((st = check_attention_sizes(cache, batch, args, false))) return st;
  if (!out_bytes) return fail(QMV_ERR_NULL, "out_bytes is NULL");
  *out_bytes = size_t(qmv::kv_attention_plan(*cache, *batch, *args).bytes);
  return ok();
}

int qmv_kv_attention(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const qmv_kv_attention_args* args, void* ws,
                     size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_attention_sizes(cache, batch, args, true))) return st;
  const qmv_kv_attention_args& a = *args;
  if (!a.q) return fail(QMV_ERR_NULL, "args->q is NULL");
  if (!a.out) return fail(QMV_ERR_NULL, "args->out is NULL");
  if (!aligned(a.q, element(a.dtype))) return fail(QMV_ERR_ALIGN, "args->q is not aligned to its element");
  if (!aligned(a.out, element(a.dtype))) return fail(QMV_ERR_ALIGN, "args->out is not aligned to its element");
  if (a.lse && !aligned(a.lse, 4)) return fail(QMV_ERR_ALIGN, "args->lse is not 4-byte aligned");
  if (!std::isfinite(a.scale)) return fail(QMV_ERR_UNSUPPORTED, "args->scale must be finite");
  if (a.out == a.q && (a.out_token != a.q_token || a.out_head != a.q_head))
    return fail(QMV_ERR_UNSUPPORTED, "args->out is q with other strides");
  if (meets_itself(batch->T, cache->D, a.q_heads, a.out_token, a.out_head))
    return fail(QMV_ERR_UNSUPPORTED, "args->out holds some values more than once");
  const Range q = reach(a.q, batch->T, a.q_heads, cache->D, a.q_token, a.q_head, a.dtype, "args->q");
  const Range out = reach(a.out, batch->T, a.q_heads, cache->D, a.out_token, a.out_head, a.dtype, "args->out");
  const Range lse{a.lse, a.lse ? 4 * batch->T * a.q_heads : 0, "args->lse"};
  if (in_cache(*cache, out)) return fail(QMV_ERR_UNSUPPORTED, "args->out lies in the cache");
  if (a.lse && in_cache(*cache, lse)) return fail(QMV_ERR_UNSUPPORTED, "args->lse lies in the cache");
  if (a.lse && ((st = check_apart(lse, q)) || (st = check_apart(lse, out)))) return st;
  const qmv::KvAttentionPlan plan = qmv::kv_attention_plan(*cache, *batch, a);
  if (plan.bytes) {
    if ((st = check_buffer(ws, "ws"))) return st;
    if (ws_bytes < size_t(plan.bytes))
      return fail(QMV_ERR_SHAPE, "ws_bytes=%llu, the call needs %lld", (unsigned long long)ws_bytes, (long long)plan.bytes);
    const Range w{ws, plan.bytes, "ws"};
    if ((st = check_apart(w, Range{cache->data, cache_bytes(*cache), "the cache"}))) return st;
    if (a.lse && (st = check_apart(w, lse))) return st;
    if ((st = check_apart(w, q)) || (st = check_apart(w, out))) return st;
  }
  if ((st = check_device())) return st;
  return launched(qmv::launch_kv_attention(*cache, *batch, a, plan, static_cast<uint8_t*>(ws), as_stream(stream)),
                  "kv_attention");
}

int qmv_rope_freqs(int64_t R, double base, const qmv_rope_scaling* scaling, float* freqs) {
  if (R < 2 || R % 2 || R > 4096) return fail(QMV_ERR_SHAPE, "R=%lld must be even, in [2, 4096]", (long long)R);
  if (!freqs) return fail(QMV_ERR_NULL, "freqs is NULL");
  if (!(std::isfinite(base) && base > 0)) return fail(QMV_ERR_UNSUPPORTED, "base must be finite and > 0");
  if (scaling) {
    const qmv_rope_scaling& c = *scaling;
    if (c.kind < QMV_ROPE_LINEAR || c.kind > QMV_ROPE_PARTS)
      return fail(QMV_ERR_UNSUPPORTED, "scaling->kind=%d is not a qmv_rope_kind", c.kind);
    if (!(std::isfinite(c.factor) && c.factor >= 1))
      return fail(QMV_ERR_UNSUPPORTED, "scaling->factor must be finite and >= 1");
    if (c.kind == QMV_ROPE_NTK) {
      if (R < 4) return fail(QMV_ERR_SHAPE, "R=%lld must be >= 4 for QMV_ROPE_NTK", (long long)R);
      base *= std::pow(c.factor, double(R) / double(R - 2));
      if (!std::isfinite(base)) return fail(QMV_ERR_UNSUPPORTED, "base stretched by scaling->factor is not finite");
    }
    if (c.kind == QMV_ROPE_PARTS &&
        !(std::isfinite(c.original) && c.original > 0 && std::isfinite(c.low) && std::isfinite(c.high) && c.low < c.high))
      return fail(QMV_ERR_UNSUPPORTED, "scaling->original must be > 0 and low < high, all finite");
  }
  // the frequencies run from 1 to this one
  if (!(std::pow(base, -2.0 * double(R / 2 - 1) / double(R)) <= 3.4028234663852886e38))
    return fail(QMV_ERR_UNSUPPORTED, "base=%g gives frequencies past the f32 range", base);
  for (int64_t i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * double(i) / double(R));
    if (scaling && scaling->kind == QMV_ROPE_LINEAR) f /= scaling->factor;
    if (scaling && scaling->kind == QMV_ROPE_PARTS) {
      const double r = scaling->original * f / 6.283185307179586;
      const double c = std::fmin(1.0, std::fmax(0.0, (r - scaling->low) / (scaling->high - scaling->low)));
      f *= c + (1.0 - c) / scaling->factor;
    }
    freqs[i] = static_cast<float>(f);
  }
  return ok();
}

int qmv_dequant(int fmt, int64_t N, int64_t K, const void* W, float* out, void* stream) {
  int st;
  if ((st = check_fmt(fmt))) return st;
  if ((st = check_shape(fmt, N, K, 1, "batch"))) return st;
  if (!W) return fail(QMV_ERR_NULL, "W is NULL");
  if (!out) return fail(QMV_ERR_NULL, "out is NULL");
  if (!aligned(W, 16)) return fail(QMV_ERR_ALIGN, "W is not 16-byte aligned");
  if (!aligned(out, 16)) return fail(QMV_ERR_ALIGN, "out is not 16-byte aligned");
  if ((N * (K / 32) + 255) / 256 >= (int64_t(1) << 31))
    return fail(QMV_ERR_OVERFLOW, "matrix too large for one dequant launch");
  if ((st = check_device())) return st;
  return launched(qmv::launch_dequant(fmt, N, K, static_cast<const uint8_t*>(W), out, as_stream(stream)),
                  "dequant");
}

}  // extern "C"
