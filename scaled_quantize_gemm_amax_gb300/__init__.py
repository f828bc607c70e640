"""FP8 scaled quantization and scaled FP8 GEMM for NVIDIA GB300 (sm_103a).

Python binding of libfp8q (C ABI in ``include/fp8q.h``).  Every step of the
path runs in the library's CUDA kernels; this module only marshals arguments
(torch tensors -> device pointers, the current torch stream) and allocates
output tensors with torch.  There is no fallback: every call raises when
``libfp8q.so`` has not been built (``scaled_quantize_gemm_amax_gb300/build.py``).
The row operators' allocation helpers do the same marshalling compiled
(``_rowops.so``, built beside the library): their calls on a few tokens last
as long as an allocation and a launch.

Entry points with the C names take tensors (or None for NULL) and raise
``FP8Error`` on a non-OK status: ``fp8_amax``, ``fp8_amax_f32``, ``fp8_compute_scale``,
``amax_history_update``, ``fp8_quantize``, ``fp8_cast_transpose``, ``fp8_cast_transpose_f32``,
``fp8_cast_transpose_multi``,
``fp8_dequantize``, ``fp8_allreduce_sum``, ``fp8_scaled_gemm``, ``fp8_scaled_gemm_amax``,
``fp8_get_device_status``, ``fp8_debug_wait_timeout``, ``fp8_debug_gemm_plan``,
``fp8_debug_index_check``; and the row operators between the linear layers,
``fp8_layer_norm``, ``fp8_layer_norm_backward``, ``fp8_gated_act``,
``fp8_gated_act_backward``, ``fp8_moe_route``, ``fp8_moe_dispatch``, ``fp8_moe_combine``,
``fp8_moe_combine_backward`` (with ``fp8_layer_norm_workspace`` and ``fp8_moe_capacity``).
``cast_transpose`` / ``dequantize`` / ``scaled_gemm`` / ``scaled_gemm_amax`` /
``layer_norm`` / ``gated_act`` / ``moe_route`` ... are allocation helpers
over them; ``linear`` holds the FP8 linear layer and the autocast scope built
on these calls, ``blocks`` the differentiable row operators and an expert MLP block.
"""
from __future__ import annotations

import ctypes
import enum
import functools
import os
import typing

import torch

__all__ = [
    "Status", "Format", "Recipe", "OutDtype", "FP8Error", "lib_path", "load_library",
    "fp8_amax", "fp8_amax_f32", "fp8_compute_scale", "amax_history_update", "fp8_quantize", "fp8_cast_transpose",
    "fp8_cast_transpose_f32",
    "fp8_cast_transpose_multi", "CastJob",
    "fp8_dequantize", "fp8_allreduce_sum", "fp8_allreduce_sum_noalloc", "fp8_scaled_gemm", "fp8_scaled_gemm_amax", "fp8_get_device_status",
    "fp8_debug_wait_timeout", "fp8_debug_gemm_plan", "fp8_debug_index_check", "fp8_status_string",
    "scale_shape", "cast_transpose", "cast_transpose_multi", "dequantize", "allreduce_sum", "scaled_gemm", "scaled_gemm_amax",
    "DelayedScaling",
    "Activation", "MoeRoute",
    "fp8_layer_norm", "fp8_layer_norm_backward", "fp8_layer_norm_workspace", "fp8_gated_act", "fp8_gated_act_backward",
    "fp8_moe_route", "fp8_moe_capacity", "fp8_moe_dispatch", "fp8_moe_combine", "fp8_moe_combine_backward",
    "layer_norm", "layer_norm_backward", "gated_act", "gated_act_backward", "moe_route", "moe_dispatch", "moe_combine",
    "moe_combine_backward", "moe_dispatch_backward",
]


class Status(enum.IntEnum):
    OK = 0
    ERR_INVALID_ARG = 1
    ERR_SHAPE = 2
    ERR_ALIGNMENT = 3
    ERR_UNSUPPORTED = 4
    ERR_CUDA = 5
    ERR_TIMEOUT = 6
    ERR_DEVICE_STATE = 7
    ERR_INDEX = 8


class Format(enum.IntEnum):
    E4M3 = 0
    E5M2 = 1


class Recipe(enum.IntEnum):
    TENSOR = 0
    BLOCK_1x128 = 1
    BLOCK_128x128 = 2
    MX_1x32 = 3
    MX_1x32_TILED = 4
    MX_1x32_FLOOR = 5          # floor-rule exponent (the alternate); layouts as MX_1x32 / MX_1x32_TILED
    MX_1x32_FLOOR_TILED = 6


class OutDtype(enum.IntEnum):
    BF16 = 0
    FP32 = 1


class Activation(enum.IntEnum):
    SILU = 0
    GELU = 1
    GELU_TANH = 2


class FP8Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = Status(status)
        super().__init__(f"{fn}: {self.status.name}")


_PKG = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_PKG, "libfp8q.so")


_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_E = ctypes.c_int
class CastJob(ctypes.Structure):
    """C layout of fp8_cast_job."""
    _fields_ = [("x", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("recipe", ctypes.c_int), ("fmt", ctypes.c_int), ("scale", ctypes.c_void_p),
                ("amax_out", ctypes.c_void_p), ("q_row", ctypes.c_void_p), ("s_row", ctypes.c_void_p),
                ("q_col", ctypes.c_void_p), ("s_col", ctypes.c_void_p)]


_SIGNATURES = {
    "fp8_amax": [_P, _I64, _I64, _P, _P],
    "fp8_amax_f32": [_P, _I64, _I64, _P, _P],
    "fp8_cast_transpose_f32": [_P, _I64, _I64, _E, _E, _P, _P, _P, _P, _P, _P, _P],
    "fp8_compute_scale": [_P, _E, _P, _P, _P],
    "amax_history_update": [_P, _I32, _P, _P, _E, _P, _P, _P],
    "fp8_cast_transpose": [_P, _I64, _I64, _E, _E, _P, _P, _P, _P, _P, _P, _P],
    "fp8_quantize": [_P, _I64, _I64, _E, _E, _P, _P, _P, _P, _P],
    "fp8_cast_transpose_multi": [_P, _I32, _P],
    "fp8_dequantize": [_P, _I64, _I64, _E, _E, _P, _P, _P],
    "fp8_allreduce_sum": [_P, _I32, _I64, _E, _P, _P, _P, _P, _P],
    "fp8_allreduce_sum_noalloc": [_P, _I32, _I64, _E, _P, _P, _P, _P],
    "fp8_scaled_gemm": [_P, _E, _E, _P, _P, _E, _E, _P, _I64, _I64, _I64, _P, _E, _P],
    "fp8_scaled_gemm_amax": [_P, _E, _E, _P, _P, _E, _E, _P, _I64, _I64, _I64, _P, _E, _P, _P, _E, _P, _P, _P],
    "fp8_layer_norm": [_P, _I64, _I64, _I64, _E, _P, _P, _E, ctypes.c_float, _P, _I64, _P, _P, _E, _P, _I64, _P, _P],
    "fp8_layer_norm_backward": [_P, _I64, _I64, _I64, _E, _P, _I64, _P, _P, _E, _P, _I64, _P, _P, _E, _P, _I64, _P, _P, _P,
                                _I64, _P],
    "fp8_layer_norm_workspace": [_I64, _I64, _P],
    "fp8_gated_act": [_P, _I64, _I64, _I64, _E, _E, _P, _I64, _P, _I64, _E, _P, _P, _P, _P, _I64, _P],
    "fp8_gated_act_backward": [_P, _I64, _I64, _I64, _E, _E, _P, _I64, _P, _I64, _E, _P, _P, _P, _P, _I64, _P, _I64, _P,
                               _I64, _P],
    "fp8_moe_route": [_P, _I32, _I64, _I32, _I32, _I32, _P, _P, _P, _I64, _P],
    "fp8_moe_capacity": [_I64, _I32, _I32, _I32, _P],
    "fp8_moe_dispatch": [_P, _I64, _I64, _I64, _E, _I32, _P, _P, _I64, _P, _I64, _P],
    "fp8_moe_combine": [_P, _I64, _I64, _I64, _E, _I64, _I32, _P, _P, _P, _I64, _P],
    "fp8_moe_combine_backward": [_P, _I64, _I64, _I64, _E, _I32, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _P],
    "fp8_get_device_status": [_P],
    "fp8_debug_wait_timeout": [_P],
    "fp8_debug_gemm_plan": [_E, _E, _E, _I64, _I64, _I64, _I32, _I32, _I32, _P],
    "fp8_debug_index_check": [_I64, _I64, _P],
    "fp8_status_string": [_E],
}


def load_library(path: str | None = None):
    """Load libfp8q.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or lib_path()
    if not os.path.exists(p):
        raise OSError(f"libfp8q.so not built at {p}; run scaled_quantize_gemm_amax_gb300/build.py")
    lib = ctypes.CDLL(p)
    for name, args in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "fp8_status_string" else ctypes.c_int
    if path is None:
        _lib = lib
    return lib


@functools.cache
def _several_gpus() -> bool:
    return torch.cuda.device_count() > 1


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    # the library launches on the current device; with one GPU there is nothing to compare
    if _several_gpus() and t.is_cuda and t.get_device() != torch.cuda.current_device():
        raise ValueError(f"a tensor on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:   # torch.cuda.current_stream().cuda_stream, without making the Stream object (4 us a call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != 0:
        raise FP8Error(fn, status)


def fp8_status_string(status: int) -> str:
    return load_library().fp8_status_string(int(status)).decode()


# ------------------------------------------------------------------ C-ABI calls
def fp8_amax(x, amax, stream=None):
    """amax[0] = max |x| (x: [rows, cols] bf16 tensor, amax: 1-float device tensor)."""
    rows, cols = (x.shape[0], x.numel() // max(x.shape[0], 1)) if x.dim() >= 1 else (1, 1)
    _check("fp8_amax", load_library().fp8_amax(_ptr(x), rows, cols, _ptr(amax), _stream(stream)))


def fp8_amax_f32(x, amax, stream=None):
    """amax[0] = max |x| of a float32 tensor."""
    rows, cols = (x.shape[0], x.numel() // max(x.shape[0], 1)) if x.dim() >= 1 else (1, 1)
    _check("fp8_amax_f32", load_library().fp8_amax_f32(_ptr(x), rows, cols, _ptr(amax), _stream(stream)))


def fp8_compute_scale(amax, fmt, scale, scale_inv, stream=None):
    _check("fp8_compute_scale",
           load_library().fp8_compute_scale(_ptr(amax), int(fmt), _ptr(scale), _ptr(scale_inv), _stream(stream)))


def amax_history_update(hist, pos, amax, fmt, scale, scale_inv, stream=None):
    _check("amax_history_update",
           load_library().amax_history_update(_ptr(hist), hist.numel(), _ptr(pos), _ptr(amax), int(fmt),
                                              _ptr(scale), _ptr(scale_inv), _stream(stream)))


def fp8_cast_transpose(x, recipe, fmt, scale, amax_out, q_row, s_row, q_col, s_col, stream=None):
    rows, cols = x.shape
    _check("fp8_cast_transpose",
           load_library().fp8_cast_transpose(_ptr(x), rows, cols, int(recipe), int(fmt), _ptr(scale),
                                             _ptr(amax_out), _ptr(q_row), _ptr(s_row), _ptr(q_col), _ptr(s_col),
                                             _stream(stream)))


def fp8_cast_transpose_f32(x, recipe, fmt, scale, amax_out, q_row, s_row, q_col, s_col, stream=None):
    rows, cols = x.shape
    _check("fp8_cast_transpose_f32",
           load_library().fp8_cast_transpose_f32(_ptr(x), rows, cols, int(recipe), int(fmt), _ptr(scale),
                                                 _ptr(amax_out), _ptr(q_row), _ptr(s_row), _ptr(q_col), _ptr(s_col),
                                                 _stream(stream)))


def fp8_cast_transpose_multi(jobs, stream=None):
    """jobs: sequence of (x, recipe, fmt, scale, amax_out, q_row, s_row, q_col, s_col), as fp8_cast_transpose."""
    arr = (CastJob * max(len(jobs), 1))()
    for i, (x, recipe, fmt, scale, amax_out, q_row, s_row, q_col, s_col) in enumerate(jobs):
        rows, cols = x.shape
        arr[i] = CastJob(_ptr(x), rows, cols, int(recipe), int(fmt), _ptr(scale), _ptr(amax_out), _ptr(q_row),
                         _ptr(s_row), _ptr(q_col), _ptr(s_col))
    _check("fp8_cast_transpose_multi",
           load_library().fp8_cast_transpose_multi(ctypes.cast(arr, ctypes.c_void_p), len(jobs), _stream(stream)))


def fp8_quantize(x, recipe, fmt, scale, amax_out, q, s, stream=None):
    rows, cols = x.shape
    _check("fp8_quantize",
           load_library().fp8_quantize(_ptr(x), rows, cols, int(recipe), int(fmt), _ptr(scale), _ptr(amax_out),
                                       _ptr(q), _ptr(s), _stream(stream)))


def fp8_dequantize(q, recipe, fmt, s, y, stream=None):
    rows, cols = q.shape
    _check("fp8_dequantize",
           load_library().fp8_dequantize(_ptr(q), rows, cols, int(recipe), int(fmt), _ptr(s), _ptr(y),
                                         _stream(stream)))


def fp8_allreduce_sum(g, fmt, amax, q, scale_inv, out, stream=None):
    k, n = g.shape
    _check("fp8_allreduce_sum",
           load_library().fp8_allreduce_sum(_ptr(g), k, n, int(fmt), _ptr(amax), _ptr(q), _ptr(scale_inv), _ptr(out),
                                            _stream(stream)))


def fp8_allreduce_sum_noalloc(g, fmt, q, scale_inv, out, stream=None):
    k, n = g.shape
    _check("fp8_allreduce_sum_noalloc",
           load_library().fp8_allreduce_sum_noalloc(_ptr(g), k, n, int(fmt), _ptr(q), _ptr(scale_inv), _ptr(out),
                                                    _stream(stream)))


def allreduce_sum(g, fmt=Format.E5M2, stream=None):
    """Allocate outputs and run fp8_allreduce_sum on g [k, n] (rank r's gradient in row r).

    Returns (out [n] fp32, q [k, n] u8, scale_inv, amax)."""
    k, n = g.shape
    dev = g.device
    amax = torch.empty(1, dtype=torch.float32, device=dev)
    q = torch.empty((k, n), dtype=torch.uint8, device=dev)
    scale_inv = torch.empty(1, dtype=torch.float32, device=dev)
    out = torch.empty(n, dtype=torch.float32, device=dev)
    fp8_allreduce_sum(g, fmt, amax, q, scale_inv, out, stream)
    return out, q, scale_inv, amax


def dequantize(q, recipe, fmt, s, stream=None):
    """Allocate y [rows, cols] bf16 and run fp8_dequantize."""
    y = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    fp8_dequantize(q, recipe, fmt, s, y, stream)
    return y


def fp8_scaled_gemm(a, fa, ra, sa, b, fb, rb, sb, c, out=OutDtype.BF16, stream=None):
    M, K = a.shape
    N = b.shape[0]
    _check("fp8_scaled_gemm",
           load_library().fp8_scaled_gemm(_ptr(a), int(fa), int(ra), _ptr(sa), _ptr(b), int(fb), int(rb), _ptr(sb),
                                          M, N, K, _ptr(c), int(out), _stream(stream)))


def fp8_scaled_gemm_amax(a, fa, ra, sa, b, fb, rb, sb, c, out, c_amax, c_scale, fc, c_q, c_scale_inv, stream=None):
    M, K = a.shape
    N = b.shape[0]
    _check("fp8_scaled_gemm_amax",
           load_library().fp8_scaled_gemm_amax(_ptr(a), int(fa), int(ra), _ptr(sa), _ptr(b), int(fb), int(rb),
                                               _ptr(sb), M, N, K, _ptr(c), int(out), _ptr(c_amax), _ptr(c_scale),
                                               int(fc), _ptr(c_q), _ptr(c_scale_inv), _stream(stream)))


# ---- row operators
def _rows(t, what: str):
    """(rows, cols, row stride) of a 2-D CUDA tensor whose rows are contiguous (one without elements is)."""
    if t.dim() == 2:
        rows, cols = t.shape
        ld, one = t.stride()
        if one == 1 or cols <= 1 or rows == 0:
            return rows, cols, ld
    raise ValueError(f"{what}: a 2-D tensor with contiguous rows is needed, not shape {tuple(t.shape)} "
                     f"stride {t.stride()}")


_DTYPE_CODE = {torch.bfloat16: 0, torch.float32: 1}


def _dtype(t, what: str) -> int:
    try:
        return _DTYPE_CODE[t.dtype]
    except KeyError:
        raise TypeError(f"{what}: bfloat16 or float32 is needed, not {t.dtype}") from None


def _like(t, ref, what: str):
    """The row stride of `t`, which must have the shape and type of `ref` (None: 0)."""
    if t is None:
        return 0
    if t.shape != ref.shape or t.dtype != ref.dtype:
        raise ValueError(f"{what}: {t.dtype} {tuple(t.shape)}, expected {ref.dtype} {tuple(ref.shape)}")
    return _rows(t, what)[2]


def _vector(t, n: int, what: str, dtype=torch.float32):
    """A dense vector (or matrix) of n elements of `dtype` (None passes)."""
    if t is not None and (t.numel() != n or t.dtype != dtype or not t.is_contiguous()):
        raise ValueError(f"{what}: {n} contiguous {dtype} elements are needed, not {t.dtype} {tuple(t.shape)}")


def _codes(q, s, rows: int, cols: int, what: str) -> int:
    """The row stride of an 8-bit copy's codes, having checked codes and multipliers (both None: 0)."""
    if q is None and s is None:
        return 0
    if q is None or s is None or q.element_size() != 1 or q.shape != (rows, cols):
        raise ValueError(f"{what}: codes [{rows}, {cols}] of one byte and their multipliers are needed")
    _vector(s, rows * ((cols + 127) // 128), f"{what} multipliers")
    return _rows(q, what)[2]


def _code_pair(qa, sa, qb, sb, rows: int, cols: int) -> int:
    """The one row stride of both 8-bit copies (each possibly None)."""
    lda, ldb = _codes(qa, sa, rows, cols, "qa"), _codes(qb, sb, rows, cols, "qb")
    if qa is not None and qb is not None and lda != ldb and rows > 1:
        raise ValueError("qa and qb: one row stride is needed for both")
    return lda or ldb


def _params(weight, bias, cols: int):
    """The type code of weight and bias (either may be None)."""
    p = weight if weight is not None else bias
    if p is None:
        return 1
    code = _dtype(p, "weight / bias")
    _vector(weight, cols, "weight", p.dtype)
    _vector(bias, cols, "bias", p.dtype)
    return code


def _on_gpu(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError(f"a CUDA tensor is needed, not one on {t.device}")


def fp8_layer_norm(x, weight, bias, eps, y, mean, rstd, fmt, q, s, stream=None):
    rows, cols, ldx = _rows(x, "x")
    dt, wdt = _dtype(x, "x"), _params(weight, bias, cols)
    ldy, ldq = _like(y, x, "y"), _codes(q, s, rows, cols, "q")
    _vector(mean, rows, "mean")
    _vector(rstd, rows, "rstd")
    _on_gpu(x, weight, bias, y, mean, rstd, q, s)
    _check("fp8_layer_norm",
           load_library().fp8_layer_norm(_ptr(x), rows, cols, ldx, dt, _ptr(weight), _ptr(bias), wdt, eps, _ptr(y), ldy,
                                         _ptr(mean), _ptr(rstd), int(fmt), _ptr(q), ldq, _ptr(s), _stream(stream)))


def fp8_layer_norm_workspace(rows: int, cols: int) -> int:
    """Bytes of fp8_layer_norm_backward's workspace (host arithmetic)."""
    n = ctypes.c_int64()
    _check("fp8_layer_norm_workspace", load_library().fp8_layer_norm_workspace(rows, cols, ctypes.addressof(n)))
    return n.value


def fp8_layer_norm_backward(dy, x, mean, rstd, fmt, q, s, weight, dx, dweight, dbias, workspace, stream=None):
    rows, cols, lddy = _rows(dy, "dy")
    dt = _dtype(dy, "dy")
    wdt = _params(weight, dweight, cols) if weight is not None or dweight is not None else _params(None, dbias, cols)
    _vector(dbias, cols, "dbias", (torch.bfloat16, torch.float32)[wdt])
    ldx, lddx, ldq = _like(x, dy, "x"), _like(dx, dy, "dx"), _codes(q, s, rows, cols, "q")
    _vector(mean, rows, "mean")
    _vector(rstd, rows, "rstd")
    _on_gpu(dy, x, mean, rstd, q, s, weight, dx, dweight, dbias, workspace)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("fp8_layer_norm_backward",
           load_library().fp8_layer_norm_backward(_ptr(dy), rows, cols, lddy, dt, _ptr(x), ldx, _ptr(mean), _ptr(rstd),
                                                  int(fmt), _ptr(q), ldq, _ptr(s), _ptr(weight), wdt, _ptr(dx), lddx,
                                                  _ptr(dweight), _ptr(dbias), _ptr(workspace), nbytes, _stream(stream)))


def fp8_gated_act(a, b, act, y, fmt, qa, sa, qb, sb, stream=None):
    rows, cols, lda = _rows(a, "a")
    ldb, ldy, dt = _like(b, a, "b"), _like(y, a, "y"), _dtype(a, "a")
    ldq = _code_pair(qa, sa, qb, sb, rows, cols)
    _on_gpu(a, b, y, qa, sa, qb, sb)
    _check("fp8_gated_act",
           load_library().fp8_gated_act(_ptr(a), rows, cols, lda, dt, int(act), _ptr(b), ldb, _ptr(y), ldy, int(fmt), _ptr(qa),
                                        _ptr(sa), _ptr(qb), _ptr(sb), ldq, _stream(stream)))


def fp8_gated_act_backward(dy, act, a, b, fmt, qa, sa, qb, sb, da, db, stream=None):
    rows, cols, lddy = _rows(dy, "dy")
    lda, ldb, dt = _like(a, dy, "a"), _like(b, dy, "b"), _dtype(dy, "dy")
    ldda, lddb = _like(da, dy, "da"), _like(db, dy, "db")
    ldq = _code_pair(qa, sa, qb, sb, rows, cols)
    _on_gpu(dy, a, b, qa, sa, qb, sb, da, db)
    _check("fp8_gated_act_backward",
           load_library().fp8_gated_act_backward(_ptr(dy), rows, cols, lddy, dt, int(act), _ptr(a), lda, _ptr(b), ldb, int(fmt),
                                                 _ptr(qa), _ptr(sa), _ptr(qb), _ptr(sb), ldq, _ptr(da), ldda, _ptr(db), lddb,
                                                 _stream(stream)))


def fp8_moe_capacity(tokens: int, k: int, n_experts: int, align: int) -> int:
    """Rows that a routing of this size can use (host arithmetic)."""
    n = ctypes.c_int64()
    _check("fp8_moe_capacity", load_library().fp8_moe_capacity(tokens, k, n_experts, align, ctypes.addressof(n)))
    return n.value


def fp8_moe_route(experts, n_experts: int, align: int, offsets, pos, src, stream=None):
    if experts.dim() != 2 or experts.dtype not in (torch.int32, torch.int64) or not experts.is_contiguous():
        raise ValueError("experts: a contiguous [tokens, k] int32 or int64 tensor is needed")
    tokens, k = experts.shape
    _vector(offsets, n_experts + 1, "offsets", torch.int32)
    _vector(pos, tokens * k, "pos", torch.int32)
    _vector(src, src.numel(), "src", torch.int32)
    _on_gpu(experts, offsets, pos, src)
    _check("fp8_moe_route",
           load_library().fp8_moe_route(_ptr(experts), 4 if experts.dtype == torch.int32 else 8, tokens, k, n_experts, align,
                                        _ptr(offsets), _ptr(pos), _ptr(src), src.numel(), _stream(stream)))


def _choices(pos, what_tokens: int | None = None):
    """(tokens, k) of a routing's pos."""
    if pos.dim() != 2 or pos.dtype != torch.int32 or not pos.is_contiguous() or what_tokens not in (None, pos.shape[0]):
        raise ValueError(f"pos: a contiguous int32 [tokens, k] tensor is needed, not {pos.dtype} {tuple(pos.shape)}"
                         + ("" if what_tokens is None else f" for {what_tokens} tokens"))
    return pos.shape


def _check_segments(out, ref, capacity: int, cols: int, what: str) -> int:
    """The row stride of a [capacity, cols] matrix of `ref`'s type."""
    if out.shape != (capacity, cols) or out.dtype != ref.dtype:
        raise ValueError(f"{what}: {ref.dtype} ({capacity}, {cols}) is needed, not {out.dtype} {tuple(out.shape)}")
    return _rows(out, what)[2]


def fp8_moe_dispatch(x, pos, src, xs, stream=None):
    tokens, cols, ldx = _rows(x, "x")
    k, dt, capacity = _choices(pos, tokens)[1], _dtype(x, "x"), src.numel()
    _vector(src, capacity, "src", torch.int32)
    ldxs = _check_segments(xs, x, capacity, cols, "xs")
    _on_gpu(x, pos, src, xs)
    _check("fp8_moe_dispatch",
           load_library().fp8_moe_dispatch(_ptr(x), tokens, cols, ldx, dt, k, _ptr(pos), _ptr(src), capacity, _ptr(xs), ldxs,
                                           _stream(stream)))


def fp8_moe_combine(ys, pos, weights, y, stream=None):
    capacity, cols, ldys = _rows(ys, "ys")
    (tokens, k), dt = _choices(pos), _dtype(ys, "ys")
    _vector(weights, tokens * k, "weights")
    ldy = _check_segments(y, ys, tokens, cols, "y")
    _on_gpu(ys, pos, weights, y)
    _check("fp8_moe_combine",
           load_library().fp8_moe_combine(_ptr(ys), capacity, cols, ldys, dt, tokens, k, _ptr(pos), _ptr(weights), _ptr(y), ldy,
                                          _stream(stream)))


def fp8_moe_combine_backward(dy, pos, src, weights, ys, dys, dweights, stream=None):
    tokens, cols, lddy = _rows(dy, "dy")
    k, dt, capacity = _choices(pos, tokens)[1], _dtype(dy, "dy"), src.numel()
    _vector(src, capacity, "src", torch.int32)
    _vector(weights, tokens * k, "weights")
    _vector(dweights, tokens * k, "dweights")
    ldys = 0 if ys is None else _check_segments(ys, dy, capacity, cols, "ys")
    lddys = _check_segments(dys, dy, capacity, cols, "dys")
    _on_gpu(dy, pos, src, weights, ys, dys, dweights)
    _check("fp8_moe_combine_backward",
           load_library().fp8_moe_combine_backward(_ptr(dy), tokens, cols, lddy, dt, k, _ptr(pos), _ptr(src), _ptr(weights),
                                                   _ptr(ys), ldys, capacity, _ptr(dys), lddys, _ptr(dweights), _stream(stream)))


def fp8_get_device_status(stream=None) -> Status:
    return Status(load_library().fp8_get_device_status(_stream(stream)))


def fp8_debug_wait_timeout(stream=None):
    _check("fp8_debug_wait_timeout", load_library().fp8_debug_wait_timeout(_stream(stream)))


def fp8_debug_index_check(index: int, extent: int, stream=None):
    _check("fp8_debug_index_check", load_library().fp8_debug_index_check(index, extent, _stream(stream)))


GEMM_VARIANTS = {0: "per-tensor", 1: "blockwise, one CTA, 128-deep stages", 3: "MXFP8",
                 4: "blockwise per-row B, one CTA", 5: "blockwise, 256-deep stages",
                 6: "blockwise per-row B, CTA pairs", 7: "blockwise, 256 x 160 pair tiles"}


def fp8_debug_gemm_plan(ra, rb, out, m: int, n: int, k: int, fused: bool = False, num_sms: int = 152,
                        resident_pairs: int = 0) -> dict:
    """The division fp8_scaled_gemm would choose (host logic only, no device call)."""
    plan = (ctypes.c_int64 * 8)()
    _check("fp8_debug_gemm_plan", load_library().fp8_debug_gemm_plan(int(ra), int(rb), int(out), m, n, k, int(fused),
                                                                      num_sms, resident_pairs, plan))
    keys = ("pair", "variant", "block_n", "tiles", "streamk", "split", "tail0", "launched")
    return dict(zip(keys, (int(v) for v in plan)))


# ------------------------------------------------------------------ allocation helpers
def scale_shape(recipe, rows: int, cols: int):
    """Shape and dtype of the multiplier array of a [rows, cols] row-wise copy."""
    recipe = Recipe(recipe)
    if recipe == Recipe.TENSOR:
        return (1,), torch.float32
    if recipe == Recipe.BLOCK_1x128:
        return (rows, cols // 128), torch.float32
    if recipe == Recipe.BLOCK_128x128:
        return (rows // 128, cols // 128), torch.float32
    if recipe in (Recipe.MX_1x32, Recipe.MX_1x32_FLOOR):
        return (rows, cols // 32), torch.uint8
    return ((rows + 127) // 128, (cols + 127) // 128, 512), torch.uint8


def cast_transpose(x, recipe, fmt, scale=None, amax_out=None, row=True, col=True, stream=None):
    """Allocate outputs with torch and run fp8_cast_transpose (bf16 x) or
    fp8_cast_transpose_f32 (float32 x).

    Returns (q_row, s_row, q_col, s_col); the parts not requested are None.
    """
    rows, cols = x.shape
    dev = x.device
    q_row = s_row = q_col = s_col = None
    if row:
        q_row = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        shp, dt = scale_shape(recipe, rows, cols)
        s_row = torch.empty(shp, dtype=dt, device=dev)
    if col:
        q_col = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
        shp, dt = scale_shape(recipe, cols, rows)
        s_col = torch.empty(shp, dtype=dt, device=dev)
    if x.dtype == torch.float32:
        fp8_cast_transpose_f32(x, recipe, fmt, scale, amax_out, q_row, s_row, q_col, s_col, stream)
    elif x.dtype == torch.bfloat16:
        fp8_cast_transpose(x, recipe, fmt, scale, amax_out, q_row, s_row, q_col, s_col, stream)
    else:
        raise TypeError(f"cast_transpose takes bfloat16 or float32 input, not {x.dtype}")
    return q_row, s_row, q_col, s_col


def cast_transpose_multi(specs, stream=None):
    """specs: sequence of (x, recipe, fmt, scale, amax_out).  Allocates every job's outputs
    with torch and runs them in one fp8_cast_transpose_multi launch; returns a list of
    (q_row, s_row, q_col, s_col) per job."""
    outs, jobs = [], []
    for x, recipe, fmt, scale, amax_out in specs:
        rows, cols = x.shape
        dev = x.device
        q_row = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        shp, dt = scale_shape(recipe, rows, cols)
        s_row = torch.empty(shp, dtype=dt, device=dev)
        q_col = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
        shp, dt = scale_shape(recipe, cols, rows)
        s_col = torch.empty(shp, dtype=dt, device=dev)
        outs.append((q_row, s_row, q_col, s_col))
        jobs.append((x, recipe, fmt, scale, amax_out, q_row, s_row, q_col, s_col))
    fp8_cast_transpose_multi(jobs, stream)
    return outs


def scaled_gemm(a, fa, ra, sa, b, fb, rb, sb, out=OutDtype.BF16, stream=None):
    """Allocate C [M, N] (bf16 or fp32) and run fp8_scaled_gemm."""
    M, N = a.shape[0], b.shape[0]
    c = torch.empty((M, N), dtype=torch.float32 if out == OutDtype.FP32 else torch.bfloat16, device=a.device)
    fp8_scaled_gemm(a, fa, ra, sa, b, fb, rb, sb, c, out, stream)
    return c


def scaled_gemm_amax(a, fa, ra, sa, b, fb, rb, sb, c_scale, fc=Format.E4M3, out=OutDtype.BF16, keep_c=True,
                     stream=None):
    """Allocate outputs and run fp8_scaled_gemm_amax.

    Returns (c or None, c_amax, c_q, c_scale_inv): C's FP8 copy with the given
    per-tensor scale (e.g. a DelayedScaling state's) and the amax of C."""
    M, N = a.shape[0], b.shape[0]
    dev = a.device
    c = None
    if keep_c:
        c = torch.empty((M, N), dtype=torch.float32 if out == OutDtype.FP32 else torch.bfloat16, device=dev)
    c_amax = torch.empty(1, dtype=torch.float32, device=dev)
    c_q = torch.empty((M, N), dtype=torch.uint8, device=dev)
    c_scale_inv = torch.empty(1, dtype=torch.float32, device=dev)
    fp8_scaled_gemm_amax(a, fa, ra, sa, b, fb, rb, sb, c, out, c_amax, c_scale, fc, c_q, c_scale_inv, stream)
    return c, c_amax, c_q, c_scale_inv


# ------------------------------------------------------------------ row operators, outputs allocated
_ext = None


def _rowops():
    """The compiled helpers (csrc/rowops_binding.cpp), bound to the loaded library."""
    global _ext
    if _ext is None:
        import importlib.machinery
        import importlib.util

        path = os.path.join(_PKG, "_rowops.so")
        if not os.path.exists(path):
            raise OSError(f"_rowops.so not built at {path}; run scaled_quantize_gemm_amax_gb300/build.py")
        lib = load_library()
        loader = importlib.machinery.ExtensionFileLoader("_rowops", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_rowops", loader))
        loader.exec_module(module)
        module.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _SIGNATURES}, FP8Error)
        _ext = module
    return _ext


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, checkpoint=None, stats: bool = True, stream=None):
    """Allocate outputs and run fp8_layer_norm on x [rows, cols].

    Returns (y, mean, rstd, q, s).  checkpoint: a Format keeps the normalised rows in 8 bits
    (q, s; else None; the codes' row stride is padded to 16 bytes).  stats=False skips mean
    and rstd (inference)."""
    return (_ext or _rowops()).layer_norm(x, weight, bias, eps, checkpoint, stats, stream)


def layer_norm_backward(dy, rstd, weight=None, x=None, mean=None, q=None, s=None, fmt=Format.E4M3, param_grads: bool = True,
                        param_dtype=None, stream=None):
    """Allocate outputs and run fp8_layer_norm_backward; x and mean, or the 8-bit copy q and s.

    Returns (dx, dweight, dbias), the last two in the weight's type (param_dtype without a
    weight; default float32), or None with param_grads=False."""
    return (_ext or _rowops()).layer_norm_backward(dy, rstd, weight, x, mean, q, s, fmt, param_grads,
                                                   param_dtype or torch.float32, stream)


def gated_act(a, b=None, act=Activation.SILU, checkpoint=None, stream=None):
    """Allocate outputs and run fp8_gated_act: f(a) * b, or f(a) without b.

    Returns (y, qa, sa, qb, sb); the 8-bit copies only with checkpoint=Format (else None; the
    codes' row stride is padded to 16 bytes)."""
    return (_ext or _rowops()).gated_act(a, b, act, checkpoint, stream)


def gated_act_backward(dy, act=Activation.SILU, a=None, b=None, qa=None, sa=None, qb=None, sb=None, fmt=Format.E4M3,
                       stream=None):
    """Allocate outputs and run fp8_gated_act_backward; a (and b), or their 8-bit copies.

    Returns (da, db): the halves of one [rows, 2 cols] tensor, or (da, None) when not gated."""
    return (_ext or _rowops()).gated_act_backward(dy, act, a, b, qa, sa, qb, sb, fmt, stream)


class MoeRoute(typing.NamedTuple):
    """Where a router's choices go: fp8_moe_route's offsets [E + 1], pos [tokens, k], src [capacity]."""
    offsets: torch.Tensor
    pos: torch.Tensor
    src: torch.Tensor


def moe_route(experts, n_experts: int, align: int = 1, stream=None) -> MoeRoute:
    """Allocate outputs and run fp8_moe_route on experts [tokens, k] (a choice outside [0, n_experts) is dropped).

    align=128 makes every expert's segment an operand of scaled_gemm."""
    return MoeRoute(*(_ext or _rowops()).moe_route(experts, n_experts, align, stream))


def moe_dispatch(x, route: MoeRoute, stream=None):
    """xs [capacity, cols]: every token's row at its choices' rows, 0 in the rows that pad."""
    return (_ext or _rowops()).moe_dispatch(x, route.pos, route.src, stream)


def moe_combine(ys, route: MoeRoute, weights=None, stream=None):
    """y [tokens, cols]: the choices' rows of ys summed with weights [tokens, k] float32 (None: 1)."""
    return (_ext or _rowops()).moe_combine(ys, route.pos, weights, stream)


def moe_combine_backward(dy, ys, route: MoeRoute, weights=None, stream=None):
    """The gradients of moe_combine: (dys [capacity, cols], dweights [tokens, k] or None without weights)."""
    return (_ext or _rowops()).moe_combine_backward(dy, ys, route.pos, route.src, weights, stream)


def moe_dispatch_backward(dxs, route: MoeRoute, stream=None):
    """The gradient of moe_dispatch: every token's choices' rows of dxs, summed."""
    return (_ext or _rowops()).moe_combine(dxs, route.pos, None, stream)


class DelayedScaling:
    """Device-resident delayed-scaling state of one tensor role (history ring,
    write position, scale, scale_inv), driven by ``amax_history_update``."""

    def __init__(self, length: int = 16, fmt=Format.E4M3, device="cuda"):
        self.fmt = Format(fmt)
        self.hist = torch.zeros(length, dtype=torch.float32, device=device)
        self.pos = torch.zeros(1, dtype=torch.int32, device=device)
        self.scale = torch.ones(1, dtype=torch.float32, device=device)
        self.scale_inv = torch.ones(1, dtype=torch.float32, device=device)
        self.amax = torch.zeros(1, dtype=torch.float32, device=device)

    def update(self, stream=None):
        """Fold self.amax (written by the cast's amax_out) into the history."""
        amax_history_update(self.hist, self.pos, self.amax, self.fmt, self.scale, self.scale_inv, stream)

    def state_dict(self):
        return {"hist": self.hist.clone(), "pos": self.pos.clone(), "scale": self.scale.clone(),
                "scale_inv": self.scale_inv.clone()}

    def load_state_dict(self, sd):
        for k in ("hist", "pos", "scale", "scale_inv"):
            getattr(self, k).copy_(sd[k])
