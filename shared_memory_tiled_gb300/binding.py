"""ctypes binding of libtranspose's C ABI (``include/transpose.h``).

Argument marshalling only: every function below forwards to the entry point
of the same name in ``_build/libtranspose.so`` and every step of the
transpose runs in the library's CUDA kernels.  Pointers are integers (device
addresses); ``stream`` is a ``cudaStream_t`` as an integer (0 = legacy
default stream), e.g. ``torch.cuda.current_stream().cuda_stream``.

The library is opened on first use.  If it has not been built, or cannot be
loaded, every call raises ``LibraryMissing``: there is no fallback path.

``transpose`` / ``copy`` and ``quantize_fp8`` / ``matmul_fp8`` / ``layernorm`` /
``layernorm_backward`` are conveniences for torch tensors: they read sizes and
pitches off the tensors' strides and call the same entry points.
"""
from __future__ import annotations

import ctypes
import enum
import os
import threading

from . import build as _build

LIB_PATH = _build.LIB_PATH

_lock = threading.Lock()
_lib = None

I64 = ctypes.c_int64
VP = ctypes.c_void_p


class Status(enum.IntEnum):
    OK = 0
    ERR_NULL = 1
    ERR_BAD_DIM = 2
    ERR_BAD_LD = 3
    ERR_OVERLAP = 4
    ERR_UNSUPPORTED = 5
    ERR_CUDA = 6
    ERR_TIMEOUT = 7


class DType(enum.IntEnum):
    F32 = 0
    BF16 = 1
    E4M3 = 2
    E5M2 = 3


class Variant(enum.IntEnum):
    AUTO = 0
    NAIVE_ROW = 1
    NAIVE_COL = 2
    TILE_PAD = 3
    TILE_VEC = 4
    TMA = 5


class Options(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("pad", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("tile_order", ctypes.c_int32), ("out_stages", ctypes.c_int32),
                ("tile_rows", ctypes.c_int32), ("tile_cols", ctypes.c_int32),
                ("schedule", ctypes.c_int32), ("threads", ctypes.c_int32)]


class Args(ctypes.Structure):
    _fields_ = [("in_", VP), ("out", VP), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("batch", I64), ("rows", I64), ("cols", I64), ("ld_in", I64), ("ld_out", I64),
                ("stride_in", I64), ("stride_out", I64), ("stream", VP)]


class Plan(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("tile_rows", ctypes.c_int32),
                ("tile_cols", ctypes.c_int32), ("threads", ctypes.c_int32),
                ("schedule", ctypes.c_int32), ("vec_in", ctypes.c_int32),
                ("vec_out", ctypes.c_int32)]


class BoundsReport(ctypes.Structure):
    _fields_ = [("refused", I64), ("first_address", ctypes.c_uint64),
                ("first_bytes", ctypes.c_int32), ("first_store", ctypes.c_int32)]


class QuantizeArgs(ctypes.Structure):
    _fields_ = [("x", VP), ("q", VP), ("scale", VP), ("qt", VP), ("scale_t", VP),
                ("x_dtype", ctypes.c_int32), ("q_dtype", ctypes.c_int32),
                ("block_rows", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("rows", I64), ("cols", I64), ("ld_x", I64), ("ld_q", I64), ("ld_scale", I64),
                ("ld_qt", I64), ("ld_scale_t", I64), ("stream", VP)]


class MatmulFp8Args(ctypes.Structure):
    _fields_ = [("a", VP), ("scale_a", VP), ("b", VP), ("scale_b", VP), ("out", VP),
                ("a_dtype", ctypes.c_int32), ("b_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("a_block_rows", ctypes.c_int32),
                ("b_block_rows", ctypes.c_int32), ("accumulate", ctypes.c_int32),
                ("m", I64), ("n", I64), ("k", I64), ("lda", I64), ("ldb", I64), ("ld_out", I64),
                ("ld_scale_a", I64), ("ld_scale_b", I64), ("stream", VP)]


class LayernormArgs(ctypes.Structure):
    _fields_ = [("x", VP), ("gamma", VP), ("beta", VP), ("y", VP), ("mean", VP), ("rstd", VP),
                ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("rows", I64),
                ("cols", I64), ("ld_x", I64), ("ld_y", I64), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("stream", VP)]


class LayernormBackwardArgs(ctypes.Structure):
    _fields_ = [("dy", VP), ("x", VP), ("gamma", VP), ("mean", VP), ("rstd", VP), ("dx", VP),
                ("dgamma", VP), ("dbeta", VP), ("workspace", VP), ("workspace_bytes", I64),
                ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("rows", I64),
                ("cols", I64), ("ld_dy", I64), ("ld_x", I64), ("ld_dx", I64), ("stream", VP)]


class LibraryMissing(RuntimeError):
    pass


class TransposeError(RuntimeError):
    def __init__(self, status: int, message: str = ""):
        self.status = Status(status) if status in Status._value2member_map_ else status
        super().__init__(f"{self.status!r}: {message}".rstrip(": "))


# Every symbol the header declares, with its ctypes signature.
SIGNATURES = {
    "tr_transpose_f32": ([VP, VP, I64, I64, I64, I64, VP], ctypes.c_int),
    "tr_transpose_bf16": ([VP, VP, I64, I64, I64, I64, VP], ctypes.c_int),
    "tr_transpose_batched_f32": ([VP, VP, I64, I64, I64, I64, I64, I64, I64, VP], ctypes.c_int),
    "tr_transpose_batched_bf16": ([VP, VP, I64, I64, I64, I64, I64, I64, I64, VP], ctypes.c_int),
    "tr_transpose_ex": ([ctypes.POINTER(Args), ctypes.POINTER(Options)], ctypes.c_int),
    "tr_copy": ([VP, VP, ctypes.c_size_t, VP], ctypes.c_int),
    "tr_transpose_inplace_f32": ([VP, I64, I64, I64, I64, VP], ctypes.c_int),
    "tr_transpose_inplace_bf16": ([VP, I64, I64, I64, I64, VP], ctypes.c_int),
    "tr_plan_variant": ([ctypes.POINTER(Args), ctypes.POINTER(Options)], ctypes.c_int32),
    "tr_plan_ex": ([ctypes.POINTER(Args), ctypes.POINTER(Options), ctypes.POINTER(Plan)],
                   ctypes.c_int),
    "tr_bank_probe": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, VP, VP], ctypes.c_int),
    "tr_operand_tiles_f32": ([VP, VP, I64, I64, I64, ctypes.c_int32, ctypes.c_int32,
                              ctypes.c_int32, VP], ctypes.c_int),
    "tr_quantize_fp8": ([ctypes.POINTER(QuantizeArgs)], ctypes.c_int),
    "tr_matmul_fp8": ([ctypes.POINTER(MatmulFp8Args)], ctypes.c_int),
    "tr_layernorm": ([ctypes.POINTER(LayernormArgs)], ctypes.c_int),
    "tr_layernorm_backward": ([ctypes.POINTER(LayernormBackwardArgs)], ctypes.c_int),
    "tr_layernorm_backward_workspace": ([I64, I64], I64),
    "tr_device_status": ([], ctypes.c_int),
    "tr_selftest_bounded_wait": ([ctypes.c_int32, I64, VP], ctypes.c_int),
    "tr_debug_bounds": ([ctypes.POINTER(BoundsReport)], ctypes.c_int),
    "tr_debug_bounds_selftest": ([ctypes.c_uint64, VP], ctypes.c_int),
    "tr_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "tr_last_error": ([], ctypes.c_char_p),
    "tr_version": ([], ctypes.c_int32),
}


def open_library(path: str):
    """Open a build of the library at ``path`` (e.g. the bounds-checked one)
    as its own ctypes handle with every entry point's signature set."""
    if not os.path.exists(path):
        raise LibraryMissing(
            f"libtranspose is not built ({path} missing); run "
            "`python -m shared_memory_tiled_gb300.build`")
    try:
        lib = ctypes.CDLL(path)
    except OSError as e:  # pragma: no cover - depends on the machine
        raise LibraryMissing(f"cannot load {path}: {e}") from e
    for name, (argtypes, restype) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = restype
    return lib


def load(path: str | None = None):
    """Open the library (once) and return the ctypes handle."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = open_library(path or LIB_PATH)
    return _lib


def _call(name, *args):
    return getattr(load(), name)(*args)


# --- the C entry points, same names ------------------------------------------------

def tr_transpose_f32(in_ptr, out_ptr, rows, cols, ld_in, ld_out, stream=0) -> int:
    return _call("tr_transpose_f32", in_ptr, out_ptr, rows, cols, ld_in, ld_out, stream)


def tr_transpose_bf16(in_ptr, out_ptr, rows, cols, ld_in, ld_out, stream=0) -> int:
    return _call("tr_transpose_bf16", in_ptr, out_ptr, rows, cols, ld_in, ld_out, stream)


def tr_transpose_batched_f32(in_ptr, out_ptr, batch, rows, cols, ld_in, ld_out, stride_in,
                             stride_out, stream=0) -> int:
    return _call("tr_transpose_batched_f32", in_ptr, out_ptr, batch, rows, cols, ld_in, ld_out,
                 stride_in, stride_out, stream)


def tr_transpose_batched_bf16(in_ptr, out_ptr, batch, rows, cols, ld_in, ld_out, stride_in,
                              stride_out, stream=0) -> int:
    return _call("tr_transpose_batched_bf16", in_ptr, out_ptr, batch, rows, cols, ld_in, ld_out,
                 stride_in, stride_out, stream)


def make_args(in_ptr, out_ptr, dtype, batch, rows, cols, ld_in, ld_out, stride_in=0,
              stride_out=0, stream=0) -> Args:
    return Args(in_ptr, out_ptr, int(dtype), 0, batch, rows, cols, ld_in, ld_out, stride_in,
                stride_out, stream)


def make_options(variant=Variant.AUTO, pad=0, ctas_per_sm=0, stages=0, tile_order=0,
                 out_stages=0, tile_rows=0, tile_cols=0, schedule=0, threads=0) -> Options:
    return Options(int(variant), pad, ctas_per_sm, stages, tile_order, out_stages, tile_rows,
                   tile_cols, schedule, threads)


def tr_transpose_ex(args: Args, opts: Options | None = None) -> int:
    return _call("tr_transpose_ex", ctypes.byref(args), ctypes.byref(opts) if opts else None)


def tr_transpose_inplace_f32(ptr, batch, n, ld, stride, stream=0) -> int:
    return _call("tr_transpose_inplace_f32", ptr, batch, n, ld, stride, stream)


def tr_transpose_inplace_bf16(ptr, batch, n, ld, stride, stream=0) -> int:
    return _call("tr_transpose_inplace_bf16", ptr, batch, n, ld, stride, stream)


def tr_copy(in_ptr, out_ptr, nbytes, stream=0) -> int:
    return _call("tr_copy", in_ptr, out_ptr, nbytes, stream)


def tr_plan_variant(args: Args, opts: Options | None = None) -> int:
    return _call("tr_plan_variant", ctypes.byref(args), ctypes.byref(opts) if opts else None)


def tr_plan_ex(args: Args, opts: Options | None, plan: Plan) -> int:
    return _call("tr_plan_ex", ctypes.byref(args), ctypes.byref(opts) if opts else None,
                 ctypes.byref(plan) if plan is not None else None)


def tr_operand_tiles_f32(a_ptr, out_ptr, m, k, lda, bm, bk, pad=-1, stream=0) -> int:
    return _call("tr_operand_tiles_f32", a_ptr, out_ptr, m, k, lda, bm, bk, pad, stream)


def tr_bank_probe(layout, reps, blocks, result_ptr, stream=0) -> int:
    return _call("tr_bank_probe", layout, reps, blocks, result_ptr, stream)


def tr_quantize_fp8(args: QuantizeArgs) -> int:
    return _call("tr_quantize_fp8", ctypes.byref(args) if args is not None else None)


def tr_matmul_fp8(args: MatmulFp8Args) -> int:
    return _call("tr_matmul_fp8", ctypes.byref(args) if args is not None else None)


def tr_layernorm(args: LayernormArgs) -> int:
    return _call("tr_layernorm", ctypes.byref(args) if args is not None else None)


def tr_layernorm_backward(args: LayernormBackwardArgs) -> int:
    return _call("tr_layernorm_backward", ctypes.byref(args) if args is not None else None)


def tr_layernorm_backward_workspace(rows, cols) -> int:
    return _call("tr_layernorm_backward_workspace", rows, cols)


def tr_selftest_bounded_wait(arrive, limit_ns, stream=0) -> int:
    return _call("tr_selftest_bounded_wait", arrive, limit_ns, stream)


def tr_debug_bounds(report: BoundsReport) -> int:
    return _call("tr_debug_bounds", ctypes.byref(report) if report is not None else None)


def tr_debug_bounds_selftest(base, stream=0) -> int:
    return _call("tr_debug_bounds_selftest", base, stream)


def tr_device_status() -> int:
    return _call("tr_device_status")


def tr_status_string(status: int) -> str:
    return _call("tr_status_string", int(status)).decode()


def tr_last_error() -> str:
    return _call("tr_last_error").decode()


def tr_version() -> int:
    return _call("tr_version")


def check(status: int) -> None:
    """Raise TransposeError for a non-OK status."""
    if status != Status.OK:
        raise TransposeError(status, f"{tr_status_string(status)}; {tr_last_error()}")


# --- torch conveniences -------------------------------------------------------------

def _dtype_of(t) -> DType:
    import torch
    if t.element_size() == 4 and t.dtype in (torch.float32, torch.int32, torch.uint32):
        return DType.F32
    if t.element_size() == 2 and t.dtype in (torch.bfloat16, torch.float16, torch.int16,
                                             torch.uint16):
        return DType.BF16
    raise TypeError(f"unsupported dtype {t.dtype}: 4-byte (fp32) or 2-byte (bf16) elements")


def _geometry(t):
    """(batch, rows, cols, ld, stride) of a 2-D or 3-D tensor with unit inner stride."""
    if t.dim() == 2:
        t = t.unsqueeze(0)
    if t.dim() != 3:
        raise ValueError("expected a 2-D or 3-D tensor")
    b, r, c = t.shape
    sb, sr, sc = t.stride()
    if c > 1 and sc != 1:
        raise ValueError("the innermost dimension must be contiguous")
    if r <= 1:
        sr = max(sr, c)
    if b <= 1:
        sb = max(sb, r * sr)
    return b, r, c, sr, sb


def transpose(x, out=None, *, variant=Variant.AUTO, pad=0, ctas_per_sm=0, stages=0,
              tile_order=0, out_stages=0, tile_rows=0, tile_cols=0, schedule=0, threads=0,
              stream=None):
    """Transpose the last two dims of a CUDA tensor ``x`` ([R, C] or [B, R, C]).

    ``out`` (optional) receives the result and may be a strided view (its row
    pitch becomes ``ld_out``); otherwise a dense output is allocated with torch.
    Launches asynchronously on ``stream`` (default: torch's current stream).
    """
    import torch
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor: the library has no CPU path")
    dt = _dtype_of(x)
    b, r, c, ld_in, s_in = _geometry(x)
    if out is None:
        shape = (c, r) if x.dim() == 2 else (b, c, r)
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    if out.dtype != x.dtype or out.device != x.device:
        raise ValueError("out must match x in dtype and device")
    ob, orr, oc, ld_out, s_out = _geometry(out)
    if (ob, orr, oc) != (b, c, r):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(b, c, r)}")
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    args = make_args(x.data_ptr(), out.data_ptr(), dt, b, r, c, ld_in, ld_out, s_in, s_out,
                     stream)
    opts = make_options(variant, pad, ctas_per_sm, stages, tile_order, out_stages, tile_rows,
                        tile_cols, schedule, threads)
    with torch.cuda.device(x.device):  # the library sets kernels up per current device
        check(tr_transpose_ex(args, opts))
    return out


def copy(src, dst, stream=None):
    """Byte copy of a contiguous CUDA tensor into another of the same byte size
    (on the same device)."""
    import torch
    if not (src.is_cuda and dst.is_cuda and src.is_contiguous() and dst.is_contiguous()):
        raise ValueError("copy wants contiguous CUDA tensors")
    n = src.numel() * src.element_size()
    if n != dst.numel() * dst.element_size():
        raise ValueError("size mismatch")
    if src.device != dst.device:
        raise ValueError("copy wants both tensors on one device")
    if stream is None:
        stream = torch.cuda.current_stream(src.device).cuda_stream
    with torch.cuda.device(src.device):
        check(tr_copy(src.data_ptr(), dst.data_ptr(), n, stream))
    return dst


def transpose_(x, stream=None):
    """Transpose the last two (equal) dims of a CUDA tensor in place."""
    import torch
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor: the library has no CPU path")
    dt = _dtype_of(x)
    b, r, c, ld, s = _geometry(x)
    if r != c:
        raise ValueError("in-place transpose needs square planes")
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    f = tr_transpose_inplace_f32 if dt == DType.F32 else tr_transpose_inplace_bf16
    with torch.cuda.device(x.device):
        check(f(x.data_ptr(), b, r, ld, s, stream))
    return x


# --- a linear layer in 8-bit floating point: torch conveniences -----------------------
#
# Kept short on the host: a call on one token costs the GPU 3-5 us, about what the
# C entry point costs the host (3-4 us), and each tensor that torch allocates costs
# 1.3-2 us, each look at a tensor or import statement 0.1-0.3 us on top.

_torch = None       # the module, once one of these functions has needed it
_KINDS: dict = {}   # {torch dtype: DType value}
_WIDE, _NARROW, _F32 = (0, 1), (2, 3), (0,)


def _need_torch():
    global _torch
    import torch
    _KINDS.update({torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2,
                   torch.float8_e5m2: 3})
    _torch = torch
    return torch


def _kind(dtype, allowed, name):
    k = _KINDS.get(dtype)
    if k not in allowed:
        raise TypeError(f"{name}: unsupported dtype {dtype}")
    return k


def _matrix(t, name, device):
    """(rows, cols, pitch) of a matrix with unit inner stride on a CUDA device."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix")
    r, c = shape
    sr, sc = t.stride()
    if sc != 1 and c > 1:
        raise ValueError(f"the innermost dimension of {name} must be contiguous")
    return r, c, (sr if r > 1 and c else max(sr, c))


def _vector(t, name, n, device):
    """Checks a contiguous vector of n values on a CUDA device."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.shape != (n,) or (t.stride(0) != 1 and n > 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}")


def _cuda(x):
    if not x.is_cuda:
        raise ValueError("expected CUDA tensors: the library has no CPU path")
    return x.device


def _run(name, args, device):
    """Calls a C entry point with its argument struct on torch's current stream
    of the device."""
    index = device.index
    # torch.cuda.current_stream(device).cuda_stream, without its 2 us of wrapping
    args.stream = _torch._C._cuda_getCurrentRawStream(index)
    f = getattr(_lib or load(), name)
    if _torch.cuda.current_device() == index:
        status = f(ctypes.byref(args))
    else:
        with _torch.cuda.device(device):  # the library sets kernels up per current device
            status = f(ctypes.byref(args))
    if status:
        check(status)


def _on(stream, x, call):
    """Makes the call, and so allocates what it returns and works in, on that
    cudaStream_t instead of torch's current stream."""
    torch = _torch or _need_torch()
    device = _cuda(x)
    s = (torch.cuda.ExternalStream(stream, device=device) if stream
         else torch.cuda.default_stream(device))
    with torch.cuda.stream(s):
        return call()


def quantize_fp8(x, *, dtype=None, block_rows=1, transposed=False, stream=None):
    """Quantize a CUDA matrix (fp32 or bf16) to 8-bit floating point.

    Returns ``(q, scale)``, and with ``transposed`` ``(q, scale, qt, scale_t)``:
    ``q`` has x's shape and ``dtype`` (torch.float8_e4m3fn, the default, or
    torch.float8_e5m2), rows padded to 16 bytes; ``scale`` is
    [ceil(cols/128), ceil(rows/block_rows)] in fp32, one scale for each block of
    block_rows (1 or 128) x 128 values, and ``q * scale`` stands for x.  ``qt``
    and ``scale_t`` are the same of x's transpose, from the same read of x.
    ``stream`` (a cudaStream_t): default torch's current stream.
    """
    if stream is not None:
        return _on(stream, x, lambda: quantize_fp8(x, dtype=dtype, block_rows=block_rows, transposed=transposed))
    torch = _torch or _need_torch()
    dev = _cuda(x)
    rows, cols, ld = _matrix(x, "x", dev)
    if dtype is None:
        dtype = torch.float8_e4m3fn
    xk, qk = _kind(x.dtype, _WIDE, "x"), _kind(dtype, _NARROW, "dtype")
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    empty, strided, f32 = torch.empty, torch.empty_strided, torch.float32
    cb, rb, ld_q = (cols + 127) // 128, (rows + block_rows - 1) // block_rows, (cols + 15) // 16 * 16
    q = strided((rows, cols), (ld_q, 1), dtype=dtype, device=dev)
    scale = empty((cb, rb), dtype=f32, device=dev)
    if not transposed:
        _run("tr_quantize_fp8", QuantizeArgs(
            x.data_ptr(), q.data_ptr(), scale.data_ptr(), None, None, xk, qk, block_rows, 0, rows,
            cols, ld, ld_q, rb, 0, 0), dev)
        return q, scale
    cbt, rbt, ld_t = (rows + 127) // 128, (cols + block_rows - 1) // block_rows, (rows + 15) // 16 * 16
    qt = strided((cols, rows), (ld_t, 1), dtype=dtype, device=dev)
    scale_t = empty((cbt, rbt), dtype=f32, device=dev)
    _run("tr_quantize_fp8", QuantizeArgs(
        x.data_ptr(), q.data_ptr(), scale.data_ptr(), qt.data_ptr(), scale_t.data_ptr(), xk, qk,
        block_rows, 0, rows, cols, ld, ld_q, rb, ld_t, rbt), dev)
    return q, scale, qt, scale_t


def _scales(scale, rows, blocks, name, device):
    """(rows to a scale, pitch): the former is told by the scales' shape."""
    kb, rb, ld = _matrix(scale, name, device)
    if kb != blocks or (rb != rows and rb != (rows + 127) // 128):
        raise ValueError(f"{name} has shape {tuple(scale.shape)}, expected "
                         f"[{blocks}, {rows} or {(rows + 127) // 128}]")
    _kind(scale.dtype, _F32, name)
    return (1 if rb == rows else 128), ld


def matmul_fp8(a, scale_a, b, scale_b, *, out=None, out_dtype=None, accumulate=False, stream=None):
    """Product ``a @ b.T`` of two 8-bit operands [m, k] and [n, k] with their scales.

    The operands are as ``quantize_fp8`` returns them (or its transposed pair):
    scales of shape [ceil(k/128), rows] hold one for each 1 x 128 values, of
    shape [ceil(k/128), ceil(rows/128)] one for each 128 x 128.  The output is
    ``out`` (fp32 or bf16, may be a strided view) or a new matrix of
    ``out_dtype`` (bf16 by default); ``accumulate`` adds to ``out``.
    ``stream`` (a cudaStream_t): default torch's current stream.
    """
    if stream is not None:
        return _on(stream, a, lambda: matmul_fp8(a, scale_a, b, scale_b, out=out, out_dtype=out_dtype,
                                                 accumulate=accumulate))
    torch = _torch or _need_torch()
    dev = _cuda(a)
    m, k, lda = _matrix(a, "a", dev)
    n, kb, ldb = _matrix(b, "b", dev)
    if kb != k:
        raise ValueError(f"a and b contract over {k} and {kb} values")
    blocks = (k + 127) // 128
    a_rows, ld_sa = _scales(scale_a, m, blocks, "scale_a", dev)
    b_rows, ld_sb = _scales(scale_b, n, blocks, "scale_b", dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an output to add to")
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
        ld_out = n
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out_dtype is not out's dtype")
        om, on, ld_out = _matrix(out, "out", dev)
        if om != m or on != n:
            raise ValueError(f"out has shape {(om, on)}, expected {(m, n)}")
    _run("tr_matmul_fp8", MatmulFp8Args(
        a.data_ptr(), scale_a.data_ptr(), b.data_ptr(), scale_b.data_ptr(), out.data_ptr(),
        _kind(a.dtype, _NARROW, "a"), _kind(b.dtype, _NARROW, "b"), _kind(out.dtype, _WIDE, "out"),
        a_rows, b_rows, 1 if accumulate else 0, m, n, k, lda, ldb, ld_out, ld_sa, ld_sb), dev)
    return out


def _like(out, x, rows, cols, dev):
    """An output of x's shape and type: (tensor, pitch)."""
    if out is None:
        return _torch.empty((rows, cols), dtype=x.dtype, device=dev), cols
    r, c, ld = _matrix(out, "out", dev)
    if r != rows or c != cols or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    return out, ld


def layernorm(x, gamma, beta=None, *, eps=1e-5, out=None, stream=None):
    """Layer norm over the rows of a CUDA matrix (fp32 or bf16).

    Returns ``(y, mean, rstd)``: y of x's type (``out`` if given), the rows'
    means and reciprocal deviations in fp32 for ``layernorm_backward`` (NaN for a
    matrix of no columns).  ``gamma`` and ``beta`` are fp32 or bf16, both the
    same.  ``stream`` (a cudaStream_t): default torch's current stream.
    """
    if stream is not None:
        return _on(stream, x, lambda: layernorm(x, gamma, beta, eps=eps, out=out))
    torch = _torch or _need_torch()
    dev = _cuda(x)
    rows, cols, ld = _matrix(x, "x", dev)
    _vector(gamma, "gamma", cols, dev)
    if beta is not None:
        _vector(beta, "beta", cols, dev)
        if beta.dtype != gamma.dtype:
            raise TypeError("gamma and beta must have the same dtype")
    xk, wk = _kind(x.dtype, _WIDE, "x"), _kind(gamma.dtype, _WIDE, "gamma")
    out, ld_y = _like(out, x, rows, cols, dev)
    empty, f32 = torch.empty, torch.float32
    mean, rstd = empty(rows, dtype=f32, device=dev), empty(rows, dtype=f32, device=dev)
    if not cols:  # the library launches nothing; the statistics of no values are 0 / 0
        mean.fill_(float("nan"))
        rstd.fill_(float("nan"))
    _run("tr_layernorm", LayernormArgs(
        x.data_ptr(), gamma.data_ptr(), None if beta is None else beta.data_ptr(), out.data_ptr(),
        mean.data_ptr(), rstd.data_ptr(), xk, wk, rows, cols, ld, ld_y, eps, 0), dev)
    return out, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd, *, bias=True, out=None, stream=None):
    """Gradients of ``layernorm``: ``(dx, dgamma, dbeta)``, dx of x's type (``out``
    if given), the others in fp32; without ``bias`` dbeta is None.  ``stream``
    (a cudaStream_t): default torch's current stream."""
    if stream is not None:
        return _on(stream, x, lambda: layernorm_backward(dy, x, gamma, mean, rstd, bias=bias, out=out))
    torch = _torch or _need_torch()
    dev = _cuda(x)
    rows, cols, ld = _matrix(x, "x", dev)
    r, c, ld_dy = _matrix(dy, "dy", dev)
    if r != rows or c != cols or dy.dtype != x.dtype:
        raise ValueError("dy must match x in shape and dtype")
    _vector(gamma, "gamma", cols, dev)
    _vector(mean, "mean", rows, dev)
    _vector(rstd, "rstd", rows, dev)
    _kind(mean.dtype, _F32, "mean")
    _kind(rstd.dtype, _F32, "rstd")
    xk, wk = _kind(x.dtype, _WIDE, "x"), _kind(gamma.dtype, _WIDE, "gamma")
    out, ld_dx = _like(out, x, rows, cols, dev)
    empty, f32 = torch.empty, torch.float32
    dgamma = empty(cols, dtype=f32, device=dev)
    dbeta = empty(cols, dtype=f32, device=dev) if bias else None
    size = (_lib or load()).tr_layernorm_backward_workspace(rows, cols)
    workspace = empty(size, dtype=torch.uint8, device=dev)
    _run("tr_layernorm_backward", LayernormBackwardArgs(
        dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        out.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr() if bias else None,
        workspace.data_ptr(), size, xk, wk, rows, cols, ld_dy, ld, ld_dx), dev)
    return out, dgamma, dbeta
