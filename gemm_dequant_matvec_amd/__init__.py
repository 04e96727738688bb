"""Python binding of libqmv: fused dequantize-and-multiply of block-quantized
weights on MI355X (gfx950).

Argument marshalling only.  Every step of the computation runs in the HIP
kernels of libqmv.so; PyTorch supplies device memory and the current stream.
Importing this package fails loudly when the library has not been built
(`python gemm_dequant_matvec_amd/build.py`); there is no CPU fallback.

    import gemm_dequant_matvec_amd as qmv
    W = qmv.pack("q4k", {"q": q, "sc": sc, "m": m, "d": d, "dmin": dmin})
    y = qmv.matvec("q4k", W, x, N, K)          # x [b][K] f32 -> y [b][N] f32
    Y = qmv.gemm("w4a16_g64", W, X, N, K)      # X [M][K] bf16 -> Y [M][N] bf16
    H, G, U = qmv.gemm_glu("q4k", Wg, Wu, X, N, K, act="silu", save=True)   # act(X Wg^T) * (X Wu^T)
    dX, dG, dU = qmv.gemm_glu_backward("q4k", Wg, Wu, G, U, dH, N, K, act="silu")
    q, k = qmv.rope(q, k, pos, qmv.rope_freqs(R))   # q [T][heads][D], k [T][kv_heads][D]
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmv.so")

FORMATS = {"q8_0": 1, "w4a16_g64": 2, "q4k": 3, "q6k": 4, "q4_0": 5, "q5_0": 6, "q5k": 7, "bf16": 8,
           "i8row": 9}
BLOCK = {"q8_0": 32, "w4a16_g64": 64, "q4k": 256, "q6k": 256, "q4_0": 32, "q5_0": 32, "q5k": 256, "bf16": 32,
         "i8row": 32}
AUX_FIELDS = {
    "q8_0": ("scale",),
    "w4a16_g64": ("scale", "zero"),
    "q4k": ("sc", "m", "d", "dmin"),
    "q6k": ("s", "d"),
    "q4_0": ("d",),
    "q5_0": ("d",),
    "q5k": ("sc", "m", "d", "dmin"),
    "bf16": (),
    "i8row": ("scale",),
}
_DTYPES = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}
# (weights per element, bytes per element) of each logical aux array
_AUX_SHAPE = {
    "q8_0": {"scale": (32, 2)},
    "w4a16_g64": {"scale": (64, 2), "zero": (64, 2)},
    "q4k": {"sc": (32, 1), "m": (32, 1), "d": (256, 2), "dmin": (256, 2)},
    "q6k": {"s": (16, 1), "d": (256, 2)},
    "q4_0": {"d": (32, 2)},
    "q5_0": {"d": (32, 2)},
    "q5k": {"sc": (32, 1), "m": (32, 1), "d": (256, 2), "dmin": (256, 2)},
    "i8row": {"scale": (None, 4)},  # one per row
}

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libqmv.so not found at {LIB_PATH}: build it with "
        "`python gemm_dequant_matvec_amd/build.py` (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)


class QmvLogical(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("aux", ctypes.c_void_p * 4)]


_i64, _vp, _int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
_lib.qmv_abi_version.argtypes = [ctypes.POINTER(ctypes.c_int)]
_lib.qmv_abi_version.restype = _int
_lib.qmv_status_string.argtypes = [_int]
_lib.qmv_status_string.restype = ctypes.c_char_p
_lib.qmv_last_error.argtypes = []
_lib.qmv_last_error.restype = ctypes.c_char_p
_lib.qmv_packed_bytes.argtypes = [_int, _i64, _i64, _i64, ctypes.POINTER(ctypes.c_size_t)]
_lib.qmv_packed_bytes.restype = _int
_lib.qmv_pack.argtypes = [_int, _i64, _i64, _i64, ctypes.POINTER(QmvLogical), _vp, _vp]
_lib.qmv_pack.restype = _int
_lib.qmv_matvec.argtypes = [_int, _i64, _i64, _i64, _vp, _vp, _int, _vp, _int, _vp]
_lib.qmv_matvec.restype = _int


class QmvEpilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p)]


_lib.qmv_matvec_ex.argtypes = [_int, _i64, _i64, _i64, _vp, _vp, _int, _vp, _int, ctypes.POINTER(QmvEpilogue), _vp]
_lib.qmv_matvec_ex.restype = _int
_lib.qmv_matvec_swiglu.argtypes = [_int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _vp, _int, _vp]
_lib.qmv_matvec_swiglu.restype = _int


class QmvMatvecItem(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("W", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("fmt", ctypes.c_int32)]


_lib.qmv_matvec_grouped.argtypes = [_int, _i64, _i64, _int, ctypes.POINTER(QmvMatvecItem), _int, _int, _vp]
_lib.qmv_matvec_grouped.restype = _int
_lib.qmv_quantize_x.argtypes = [_i64, _i64, _vp, _vp, _vp]
_lib.qmv_quantize_x.restype = _int
_lib.qmv_q8x_bytes.argtypes = [_i64, _i64, ctypes.POINTER(ctypes.c_size_t)]
_lib.qmv_q8x_bytes.restype = _int
_lib.qmv_gemm.argtypes = [_int, _i64, _i64, _i64, _vp, _vp, _int, _vp, _int, _vp]
_lib.qmv_gemm.restype = _int
_lib.qmv_gemm_glu.argtypes = [_int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _int, _vp, _int, _vp, _vp, _vp]
_lib.qmv_gemm_glu.restype = _int
_lib.qmv_gemm_glu_backward.argtypes = [_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _int, _int, _vp, _vp, _vp, _vp,
                                       ctypes.c_size_t, _vp]
_lib.qmv_gemm_glu_backward.restype = _int
_lib.qmv_gemm_glu_backward_bytes.argtypes = [_int, _i64, _i64, _i64, ctypes.POINTER(ctypes.c_size_t)]
_lib.qmv_gemm_glu_backward_bytes.restype = _int
_lib.qmv_gemm_glu_backward_ex.argtypes = [_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _vp, _vp,
                                          _vp, _vp, ctypes.c_size_t, _vp]
_lib.qmv_gemm_glu_backward_ex.restype = _int
_lib.qmv_gemm_glu_backward_ex_bytes.argtypes = [_int, _i64, _i64, _i64, _int, ctypes.POINTER(ctypes.c_size_t)]
_lib.qmv_gemm_glu_backward_ex_bytes.restype = _int


class QmvRopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("x_token", ctypes.c_int64), ("x_head", ctypes.c_int64),
                ("y_token", ctypes.c_int64), ("y_head", ctypes.c_int64)]


class QmvRopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("original", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double)]


_lib.qmv_rope.argtypes = [_i64, _i64, _i64, _int, _int, _vp, _int, _vp, _vp, ctypes.c_float,
                          _int, _vp]
_lib.qmv_rope.restype = _int
_lib.qmv_rope_freqs.argtypes = [_i64, ctypes.c_double, ctypes.POINTER(QmvRopeScaling), ctypes.POINTER(ctypes.c_float)]
_lib.qmv_rope_freqs.restype = _int
_lib.qmv_dequant.argtypes = [_int, _i64, _i64, _vp, _vp, _vp]
_lib.qmv_dequant.restype = _int

EXPORTS = ("qmv_abi_version", "qmv_status_string", "qmv_last_error", "qmv_packed_bytes",
           "qmv_pack", "qmv_matvec", "qmv_matvec_ex", "qmv_matvec_swiglu", "qmv_matvec_grouped", "qmv_gemm",
           "qmv_dequant", "qmv_quantize_x", "qmv_q8x_bytes")
LAYER_EXPORTS = ("qmv_gemm_glu", "qmv_gemm_glu_backward", "qmv_gemm_glu_backward_bytes", "qmv_gemm_glu_backward_ex",
                 "qmv_gemm_glu_backward_ex_bytes", "qmv_rope", "qmv_rope_freqs")


class QmvError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_lib.qmv_status_string(status).decode()} ({status}): {message}")


def _check(status: int) -> None:
    if status != 0:
        raise QmvError(status, _lib.qmv_last_error().decode())


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        if fmt not in FORMATS:
            raise ValueError(f"unknown format {fmt!r}; one of {sorted(FORMATS)}")
        return FORMATS[fmt]
    return int(fmt)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _need(t: torch.Tensor, nbytes: int, what: str) -> None:
    """The C ABI sees only pointers: a buffer shorter than the call will touch
    is rejected here, before anything reaches the device."""
    if _nbytes(t) < nbytes:
        raise ValueError(f"{what} holds {_nbytes(t)} bytes, the call needs {nbytes}")


def _need_dtype(t: torch.Tensor, dtype: torch.dtype, what: str) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libqmv must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libqmv must be contiguous")
    return t.data_ptr()


def abi_version() -> tuple[int, int]:
    lv = ctypes.c_int(0)
    v = _lib.qmv_abi_version(ctypes.byref(lv))
    return v, lv.value


def packed_bytes(fmt, N: int, K: int, batch: int = 1) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.qmv_packed_bytes(_fmt(fmt), N, K, batch, ctypes.byref(out)))
    return out.value


def pack(fmt, logical: dict, N: int | None = None, K: int | None = None, batch: int = 1,
         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Pack logical device arrays (dict of tensors named as in AUX_FIELDS plus "q")."""
    name = fmt if isinstance(fmt, str) else {v: k for k, v in FORMATS.items()}[fmt]
    q = logical["q"]
    if N is None or K is None:
        N, K = q.shape[-2], q.shape[-1]
    nbytes = packed_bytes(name, N, K, batch)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _need(out, nbytes, "out")
    _need(q, batch * N * K * (2 if name == "bf16" else 1), "q")
    for field in AUX_FIELDS[name]:
        if field not in logical:
            raise ValueError(f"{name} needs the logical array {field!r}")
        per = _AUX_SHAPE[name][field]
        _need(logical[field], batch * N * (K // per[0] if per[0] else 1) * per[1], field)
    src = QmvLogical()
    src.q = _ptr(q)
    for i, field in enumerate(AUX_FIELDS[name]):
        src.aux[i] = _ptr(logical[field])
    _check(_lib.qmv_pack(_fmt(name), N, K, batch, ctypes.byref(src), _ptr(out), _stream(stream)))
    return out


class Q8X:
    """Activations quantized to 8-bit blocks by quantize_x: `data` is the
    device buffer (uint8), `K` and `batch` its shape."""

    def __init__(self, data: torch.Tensor, K: int, batch: int):
        self.data, self.K, self.batch = data, K, batch


def q8x_bytes(K: int, batch: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.qmv_q8x_bytes(K, batch, ctypes.byref(out)))
    return out.value


def quantize_x(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> Q8X:
    """f32 x [b][K] -> Q8X (per 32 activations: 8-bit codes and an f32 scale)."""
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    b, K = x2.shape
    nbytes = q8x_bytes(K, b)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    _need_dtype(x2, torch.float32, "x")
    _need(out, nbytes, "out")
    _check(_lib.qmv_quantize_x(K, b, _ptr(x2), _ptr(out), _stream(stream)))
    return Q8X(out, K, b)


def _xarg(x, K: int):
    """(pointer, dtype code, batch) of an activation argument: a tensor [b][K]
    (f32 / f16) or a Q8X."""
    if isinstance(x, Q8X):
        if x.K != K:
            raise ValueError(f"Q8X activations have K={x.K}, expected K={K}")
        _need(x.data, q8x_bytes(K, x.batch), "x")
        return _ptr(x.data), 4, x.batch, x.data.device
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    if x2.shape[1] != K:
        raise ValueError(f"x has {x2.shape[1]} columns, expected K={K}")
    if x2.dtype not in _DTYPES:
        raise ValueError("x dtype must be float32, float16 or bfloat16")
    return _ptr(x2), _DTYPES[x2.dtype], x2.shape[0], x2.device


def matvec(fmt, W: torch.Tensor, x, N: int, K: int, y: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """y [b][N] f32 = W x for x [b][K] (f32, f16 for w4a16_g64, or a Q8X from quantize_x)."""
    b = x.batch if isinstance(x, Q8X) else (x.shape[0] if x.dim() == 2 else 1)
    dev = x.data.device if isinstance(x, Q8X) else x.device
    if y is None:
        y = torch.empty((b, N), dtype=torch.float32, device=dev)
    if y.dtype not in _DTYPES:
        raise ValueError("y dtype must be float32, float16 or bfloat16")
    _need(W, packed_bytes(fmt, N, K), "W")
    _need(y, b * N * 4, "y")
    xp, xdt, b, _ = _xarg(x, K)
    _check(_lib.qmv_matvec(_fmt(fmt), N, K, b, _ptr(W), xp, xdt, _ptr(y), _DTYPES[y.dtype], _stream(stream)))
    return y


def matvec_ex(fmt, W: torch.Tensor, x: torch.Tensor, N: int, K: int, y: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [b][N] f32 = residual + (W x + bias): the bias / residual add fused into
    the matvec.  bias f32 [N] or None; residual f32 [b][N] or None (may be y).
    x as in matvec."""
    b = x.batch if isinstance(x, Q8X) else (x.shape[0] if x.dim() == 2 else 1)
    dev = x.data.device if isinstance(x, Q8X) else x.device
    if y is None:
        y = torch.empty((b, N), dtype=torch.float32, device=dev)
    if y.dtype not in _DTYPES:
        raise ValueError("y dtype must be float32, float16 or bfloat16")
    _need(W, packed_bytes(fmt, N, K), "W")
    _need(y, b * N * 4, "y")
    if bias is not None:
        _need_dtype(bias, torch.float32, "bias")
        _need(bias, N * 4, "bias")
    if residual is not None:
        _need_dtype(residual, torch.float32, "residual")
        _need(residual, b * N * 4, "residual")
    xp, xdt, b, _ = _xarg(x, K)  # every size check above: pointers only from here on
    ep = QmvEpilogue()
    ep.bias = _ptr(bias)
    ep.residual = _ptr(residual)
    _check(_lib.qmv_matvec_ex(_fmt(fmt), N, K, b, _ptr(W), xp, xdt, _ptr(y),
                              _DTYPES[y.dtype], ctypes.byref(ep), _stream(stream)))
    return y


def matvec_swiglu(fmt, W_gate: torch.Tensor, W_up: torch.Tensor, x: torch.Tensor, N: int, K: int,
                  h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h [b][N] f32 = silu(W_gate x) * (W_up x), gate / up / SwiGLU in one pass
    (x as in matvec)."""
    b = x.batch if isinstance(x, Q8X) else (x.shape[0] if x.dim() == 2 else 1)
    dev = x.data.device if isinstance(x, Q8X) else x.device
    if h is None:
        h = torch.empty((b, N), dtype=torch.float32, device=dev)
    if h.dtype not in _DTYPES:
        raise ValueError("h dtype must be float32, float16 or bfloat16")
    _need(W_gate, packed_bytes(fmt, N, K), "W_gate")
    _need(W_up, packed_bytes(fmt, N, K), "W_up")
    _need(h, b * N * 4, "h")
    xp, xdt, b, _ = _xarg(x, K)
    _check(_lib.qmv_matvec_swiglu(_fmt(fmt), N, K, b, _ptr(W_gate), _ptr(W_up), xp, xdt,
                                  _ptr(h), _DTYPES[h.dtype], _stream(stream)))
    return h


def matvec_grouped(fmt, items, K: int, stream=None) -> list:
    """Several matvecs of one K in as few launches as possible.

    items: sequence of (W, x, N), (W, x, N, y) or (W, x, N, y, item_fmt); x
    [b][K] (same b and dtype for all) or a Q8X of b vectors (then for all), y
    allocated as f32 [b][N] when absent or None; item_fmt overrides fmt for
    that matrix (fmt may then be None).  Returns the list of y.
    """
    arr = (QmvMatvecItem * len(items))()
    outs, rows = [], []
    b = xdt = None
    for i, it in enumerate(items):  # every size check before any pointer is taken
        W, x, N = it[0], it[1], it[2]
        if isinstance(x, Q8X):
            if x.K != K:
                raise ValueError(f"items[{i}]: Q8X activations have K={x.K}, expected K={K}")
            _need(x.data, q8x_bytes(K, x.batch), f"items[{i}].x")
            x2, shape, dt, device = x.data, (x.batch, K), "q8x", x.data.device
        else:
            x2 = x if x.dim() == 2 else x.reshape(1, -1)
            shape, dt, device = tuple(x2.shape), x2.dtype, x.device
            if dt not in _DTYPES:
                raise ValueError("x dtype must be float32, float16 or bfloat16")
        if b is None:
            b, xdt = shape[0], dt
        if shape != (b, K) or dt != xdt:
            raise ValueError("all items need x of shape [b][K] and one dtype")
        y = it[3] if len(it) > 3 and it[3] is not None else torch.empty((b, N), dtype=torch.float32,
                                                                          device=device)
        ifmt = it[4] if len(it) > 4 and it[4] is not None else fmt
        if ifmt is None:
            raise ValueError(f"item {i} names no format and the call's fmt is None")
        _need(W, packed_bytes(ifmt, N, K), f"items[{i}].W")
        _need(y, b * N * 4, f"items[{i}].y")
        rows.append((W, x2, N, y, it[4] if len(it) > 4 else None))
        outs.append(y)
    for i, (W, x2, N, y, ifmt) in enumerate(rows):
        arr[i].N, arr[i].W, arr[i].x, arr[i].y = N, _ptr(W), _ptr(x2), _ptr(y)
        arr[i].fmt = _fmt(ifmt) if ifmt is not None else 0
    _check(_lib.qmv_matvec_grouped(0 if fmt is None else _fmt(fmt), K, b, len(items), arr,
                                   4 if xdt == "q8x" else _DTYPES[xdt],
                                   _DTYPES[torch.float32], _stream(stream)))
    return outs


def gemm(fmt, W: torch.Tensor, X: torch.Tensor, N: int, K: int, Y: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Y [M][N] bf16 = X W^T for X [M][K] bf16, on the matrix cores."""
    M = X.shape[0]
    if X.shape[1] != K:
        raise ValueError(f"X has {X.shape[1]} columns, expected K={K}")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if X.dtype not in _DTYPES or Y.dtype not in _DTYPES:
        raise ValueError("X / Y dtype must be float32, float16 or bfloat16")
    _need(W, packed_bytes(fmt, N, K), "W")
    _need(Y, M * N * Y.element_size(), "Y")
    _check(_lib.qmv_gemm(_fmt(fmt), N, K, M, _ptr(W), _ptr(X), _DTYPES[X.dtype], _ptr(Y),
                         _DTYPES[Y.dtype], _stream(stream)))
    return Y


GLU_UNROUNDED = 1  # qmv_glu_flags
ACTS = {"silu": 1, "gelu_tanh": 2, "gelu": 3}
ROPE_LAYOUTS = {"half": 1, "interleaved": 2}
ROPE_KINDS = {"linear": 1, "ntk": 2, "parts": 3}

# The many-token operators below are called once or twice per layer, for single
# tokens too: their checks are kept to attribute reads (sizes are cached, the
# stream comes as a raw handle), a few microseconds per call.
#
# stream= runs a call there, like every call's: the caller has that stream wait for
# the work that fills the tensors, and keeps the tensors, or tells the allocator
# (Tensor.record_stream), until it is done.  What a call allocates itself belongs to
# that stream.
_packed_bytes_cached = functools.lru_cache(maxsize=4096)(packed_bytes)


def _act(act) -> int:
    if isinstance(act, str):
        if act not in ACTS:
            raise ValueError(f"unknown activation {act!r}; one of {sorted(ACTS)}")
        return ACTS[act]
    return int(act)


def _on_current_device(t: torch.Tensor) -> int:
    """The raw current stream, for a call whose tensors are on t's device, which
    has to be the current one: kernels are launched there."""
    if not t.is_cuda:
        raise ValueError("tensors passed to libqmv must live on the GPU")
    device = t.get_device()
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on device {device}, the current device is {torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(device)


def _no_gradient(what: str, *tensors) -> None:
    """The calls below record nothing for autograd: a result of tensors that want a
    gradient would lose it without a word."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError(f"{what} records no gradient, and a tensor passed to it requires one: call it under "
                                 "torch.no_grad() or in an autograd function, or pass it detached")


def _written(*tensors) -> None:
    """Tells autograd that the caller's own tensors were written to, as torch's
    in-place operations do: a backward pass that saved one of them then refuses to
    run on the new values."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _weight(W: torch.Tensor, nbytes: int, device: int, what: str) -> int:
    """Pointer of a packed matrix."""
    if W.nbytes < nbytes:
        raise ValueError(f"{what} holds {W.nbytes} bytes, the call needs {nbytes}")
    if not W.is_contiguous():
        raise ValueError("tensors passed to libqmv must be contiguous")
    if W.get_device() != device:
        raise ValueError(f"{what} is on {W.device}, the call's tensors on device {device}")
    return W.data_ptr()


def _like(t: torch.Tensor | None, like: torch.Tensor, shape: tuple, what: str) -> torch.Tensor:
    """t, or a new tensor in its place: of this shape, contiguous, of like's dtype and device."""
    if t is None:
        return torch.empty_like(like) if like.shape == shape else like.new_empty(shape)
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype != like.dtype:
        raise ValueError(f"{what} must be {like.dtype}, got {t.dtype}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{what} is on {t.device}, expected {like.device}")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libqmv must be contiguous")
    return t


def gemm_glu(fmt, W_gate: torch.Tensor, W_up: torch.Tensor, X: torch.Tensor, N: int, K: int, act="silu",
             H: torch.Tensor | None = None, G: torch.Tensor | None = None, U: torch.Tensor | None = None,
             save: bool = False, stream=None):
    """H [M][N] = act(X W_gate^T) * (X W_up^T) for X [M][K] (bf16 or f16, as H), in one kernel.

    act: "silu", "gelu_tanh" or "gelu".  With save=True (or G and U given) the
    two products are kept for gemm_glu_backward and (H, G, U) is returned.
    Nothing is recorded for autograd: where gradients are enabled, tensors that
    require one are refused (here and in the two functions below).
    """
    if stream is not None:  # what is allocated here belongs to that stream too
        with torch.cuda.stream(stream):
            return gemm_glu(fmt, W_gate, W_up, X, N, K, act, H, G, U, save)
    _no_gradient("gemm_glu", X, H, G, U)
    if X.dim() != 2 or X.shape[1] != K:
        raise ValueError(f"X has shape {tuple(X.shape)}, expected [M][{K}]")
    if X.dtype not in _DTYPES:
        raise ValueError("X dtype must be float32, float16 or bfloat16")
    if (G is None) != (U is None):
        raise ValueError("G and U go together")
    shape, dt, f, a = (X.shape[0], N), _DTYPES[X.dtype], _fmt(fmt), _act(act)
    s, device = _on_current_device(X), X.get_device()
    nbytes = _packed_bytes_cached(f, N, K)
    wg, wu = _weight(W_gate, nbytes, device, "W_gate"), _weight(W_up, nbytes, device, "W_up")
    if not X.is_contiguous():
        raise ValueError("tensors passed to libqmv must be contiguous")
    given = H, G, U
    H = _like(H, X, shape, "H")
    if not save and G is None:
        _check(_lib.qmv_gemm_glu(f, N, K, shape[0], wg, wu, X.data_ptr(), dt, a, H.data_ptr(), dt, None, None, s))
        _written(*given)
        return H
    G, U = _like(G, X, shape, "G"), _like(U, X, shape, "U")
    _check(_lib.qmv_gemm_glu(f, N, K, shape[0], wg, wu, X.data_ptr(), dt, a, H.data_ptr(), dt, G.data_ptr(),
                             U.data_ptr(), s))
    _written(*given)
    return H, G, U


def gemm_glu_backward_bytes(fmt, N: int, K: int, M: int, unrounded: bool = False) -> int:
    """Bytes of scratch memory that gemm_glu_backward needs for these sizes."""
    out = ctypes.c_size_t(0)
    _check(_lib.qmv_gemm_glu_backward_ex_bytes(_fmt(fmt), N, K, M, GLU_UNROUNDED if unrounded else 0, ctypes.byref(out)))
    return out.value


_backward_bytes_cached = functools.lru_cache(maxsize=4096)(gemm_glu_backward_bytes)


def gemm_glu_backward(fmt, W_gate: torch.Tensor, W_up: torch.Tensor, G: torch.Tensor, U: torch.Tensor,
                      dH: torch.Tensor, N: int, K: int, act="silu", dG: torch.Tensor | None = None,
                      dU: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None, unrounded: bool = False):
    """(dX [M][K], dG [M][N], dU [M][N]) of gemm_glu for the gradient dH [M][N] of H,
    from its saved G and U; all of one dtype.  dX is the sum over the returned
    dG and dU, which are rounded to that type; with unrounded=True over their
    values before that rounding, at twice the matrix operations and without its
    error.  dG and dU may be given as two of the buffers G, U and dH.  workspace:
    scratch memory of gemm_glu_backward_bytes bytes (of the same unrounded),
    allocated when absent."""
    if stream is not None:  # what is allocated here belongs to that stream too
        with torch.cuda.stream(stream):
            return gemm_glu_backward(fmt, W_gate, W_up, G, U, dH, N, K, act, dG, dU, dX, workspace, None, unrounded)
    _no_gradient("gemm_glu_backward", G, U, dH, dG, dU, dX)
    if G.dtype not in _DTYPES:
        raise ValueError("G dtype must be float32, float16 or bfloat16")
    shape, f, a = (G.shape[0], N), _fmt(fmt), _act(act)
    M = shape[0]
    _like(G, G, shape, "G")
    _like(U, G, shape, "U")
    _like(dH, G, shape, "dH")
    s, device = _on_current_device(G), G.get_device()
    nbytes = _packed_bytes_cached(f, N, K)
    wg, wu = _weight(W_gate, nbytes, device, "W_gate"), _weight(W_up, nbytes, device, "W_up")
    given = dG, dU, dX, workspace
    dG, dU, dX = _like(dG, G, shape, "dG"), _like(dU, G, shape, "dU"), _like(dX, G, (M, K), "dX")
    unrounded = bool(unrounded)
    nbytes = _backward_bytes_cached(f, N, K, M, unrounded)
    ws = None
    if nbytes:
        if workspace is None:
            workspace = G.new_empty(nbytes, dtype=torch.uint8)
        ws = _weight(workspace, nbytes, device, "workspace")
    _check(_lib.qmv_gemm_glu_backward_ex(f, N, K, M, wg, wu, G.data_ptr(), U.data_ptr(), dH.data_ptr(),
                                         _DTYPES[G.dtype], a, GLU_UNROUNDED if unrounded else 0, dG.data_ptr(),
                                         dU.data_ptr(), dX.data_ptr(), ws, nbytes, s))
    _written(*given)
    return dX, dG, dU


def rope_freqs(R: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0, original: float = 0.0,
               low: float = 1.0, high: float = 32.0, device="cuda") -> torch.Tensor:
    """The R/2 rotary frequencies base^(-2i/R) as f32, stretched for a longer
    context by scaling: "linear" (all divided by factor), "ntk" (a larger base)
    or "parts" (pairs with fewer than `low` turns over the `original` context
    divided by factor, those with more than `high` kept, a ramp between)."""
    host = torch.empty(max(0, R // 2), dtype=torch.float32)
    sc = None
    if scaling is not None:
        if scaling not in ROPE_KINDS:
            raise ValueError(f"unknown scaling {scaling!r}; one of {sorted(ROPE_KINDS)}")
        sc = ctypes.byref(QmvRopeScaling(ROPE_KINDS[scaling], factor, original, low, high))
    _check(_lib.qmv_rope_freqs(R, base, sc, ctypes.cast(host.data_ptr(), ctypes.POINTER(ctypes.c_float))))
    return host.to(device)


_RopeFields = {7: struct.Struct("7q"), 14: struct.Struct("14q")}  # qmv_rope_tensor: seven 8-byte fields


def _rope_out(x: torch.Tensor, y: torch.Tensor | None, what: str) -> torch.Tensor:
    if y is None:
        return torch.empty_like(x)
    if y.shape != x.shape or y.dtype != x.dtype or y.get_device() != x.get_device():
        raise ValueError(f"{what}_out must have {what}'s shape, dtype and device")
    if any(n > 1 and st == 0 for n, st in zip(y.shape, y.stride())):
        raise ValueError(f"{what}_out holds some values more than once")
    return y


def _rope_fields(x: torch.Tensor, y: torch.Tensor, what: str) -> tuple:
    (xt, xh, xd), (yt, yh, yd) = x.stride(), y.stride()
    if (xd != 1 or yd != 1) and x.shape[2] > 1:
        raise ValueError(f"the values of a head of {what} must be adjacent")
    return x.data_ptr(), y.data_ptr(), x.shape[1], xt, xh, yt, yh


def rope(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, freqs: torch.Tensor, layout="half",
         amplitude: float = 1.0, inverse: bool = False, q_out: torch.Tensor | None = None,
         k_out: torch.Tensor | None = None, stream=None):
    """Rotary positions of q [T][heads][D] and k [T][kv_heads][D] (or None) at pos
    int64 [T], in one launch; returns (q_out, k_out).

    freqs f32 [R/2] names the frequencies of the first R values of every head
    (the rest is copied); layout "half" pairs (i, i + R/2), "interleaved"
    (2i, 2i + 1).  The cosines and sines are multiplied by amplitude.
    inverse=True turns back: the gradient of the forward call.  q and k may be
    strided (slices of one fused product) as long as a head's values are
    adjacent; q_out=q, k_out=k works in place.
    """
    if stream is not None:  # what is allocated here belongs to that stream too
        with torch.cuda.stream(stream):
            return rope(q, k, pos, freqs, layout, amplitude, inverse, q_out, k_out)
    _no_gradient("rope", q, k, freqs, q_out, k_out)
    if layout in ROPE_LAYOUTS:
        layout = ROPE_LAYOUTS[layout]
    elif isinstance(layout, str):
        raise ValueError(f"unknown layout {layout!r}; one of {sorted(ROPE_LAYOUTS)}")
    if q.dim() != 3:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [T][heads][D]")
    T, _, D = q.shape
    if q.dtype not in _DTYPES:
        raise ValueError("q dtype must be float32, float16 or bfloat16")
    _need_dtype(pos, torch.int64, "pos")
    _need_dtype(freqs, torch.float32, "freqs")
    if pos.numel() != T:
        raise ValueError(f"pos holds {pos.numel()} positions, q {T} tokens")
    if k is None and k_out is not None:
        raise ValueError("k_out is given without k")
    if k is not None and (k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or k.dtype != q.dtype):
        raise ValueError(f"k has shape {tuple(k.shape)} and {k.dtype}, expected [{T}][heads][{D}] and {q.dtype}")
    s, device = _on_current_device(q), q.get_device()
    if pos.get_device() != device or freqs.get_device() != device or (k is not None and k.get_device() != device):
        raise ValueError("q, k, pos and freqs must be on one device")
    if not (pos.is_contiguous() and freqs.is_contiguous()):
        raise ValueError("tensors passed to libqmv must be contiguous")
    given = q_out, k_out
    q_out = _rope_out(q, q_out, "q")
    fields = _rope_fields(q, q_out, "q")
    if k is not None:
        k_out = _rope_out(k, k_out, "k")
        fields += _rope_fields(k, k_out, "k")
    _check(_lib.qmv_rope(T, D, 2 * freqs.numel(), layout, len(fields) // 7, _RopeFields[len(fields)].pack(*fields),
                         _DTYPES[q.dtype],
                         pos.data_ptr(), freqs.data_ptr(), amplitude, inverse, s))
    _written(*given)
    return q_out, None if k is None else k_out


def dequant(fmt, W: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """Dense f32 [N][K] copy of a packed matrix (bit-exact; inspection/testing)."""
    if out is None:
        out = torch.empty((N, K), dtype=torch.float32, device=W.device)
    _need(W, packed_bytes(fmt, N, K), "W")
    _need_dtype(out, torch.float32, "out")
    _need(out, N * K * 4, "out")
    _check(_lib.qmv_dequant(_fmt(fmt), N, K, _ptr(W), _ptr(out), _stream(stream)))
    return out


def raw_call(name: str, *args) -> int:
    """Call a C entry point with raw arguments (tests of the ABI's error paths)."""
    return getattr(_lib, name)(*args)


def last_error() -> str:
    return _lib.qmv_last_error().decode()
