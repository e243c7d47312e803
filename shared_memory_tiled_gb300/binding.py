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
import functools
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

_TORCH_TYPES: dict = {}


def _torch_types() -> dict:
    """{torch dtype: DType} of the linear layer's operators."""
    if not _TORCH_TYPES:
        import torch
        _TORCH_TYPES.update({torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2,
                             torch.float8_e5m2: 3})
    return _TORCH_TYPES


def _type(t, name, allowed):
    d = _torch_types().get(t.dtype)
    if d not in allowed:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return d


def _matrix(t, name, device=None):
    """(rows, cols, pitch) of a CUDA matrix with unit inner stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor: the library has no CPU path")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    r, c = t.shape
    sr, sc = t.stride()
    if c > 1 and sc != 1:
        raise ValueError(f"the innermost dimension of {name} must be contiguous")
    return r, c, (sr if r > 1 else max(sr, c))


def _vector(t, name, n, device):
    """Checks a contiguous CUDA vector of n values."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}")


def _run(fn, args, device):
    """Calls a C entry point with its argument struct on torch's current stream
    of the device."""
    import torch
    args.stream = torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() == device.index:
        check(fn(args))
    else:
        with torch.cuda.device(device):  # the library sets kernels up per current device
            check(fn(args))


def _on_stream(f):
    """``stream=``: the call, and the allocation of what it returns and works in,
    happens on that cudaStream_t instead of torch's current stream."""
    @functools.wraps(f)
    def call(x, *args, stream=None, **kw):
        if stream is None:
            return f(x, *args, **kw)
        import torch
        if not x.is_cuda:
            raise ValueError("expected CUDA tensors: the library has no CPU path")
        s = (torch.cuda.ExternalStream(stream, device=x.device) if stream
             else torch.cuda.default_stream(x.device))
        with torch.cuda.stream(s):
            return f(x, *args, **kw)
    return call


@_on_stream
def quantize_fp8(x, *, dtype=None, block_rows=1, transposed=False):
    """Quantize a CUDA matrix (fp32 or bf16) to 8-bit floating point.

    Returns ``(q, scale)``, and with ``transposed`` ``(q, scale, qt, scale_t)``:
    ``q`` has x's shape and ``dtype`` (torch.float8_e4m3fn, the default, or
    torch.float8_e5m2), rows padded to 16 bytes; ``scale`` is
    [ceil(cols/128), ceil(rows/block_rows)] in fp32, one scale for each block of
    block_rows (1 or 128) x 128 values, and ``q * scale`` stands for x.  ``qt``
    and ``scale_t`` are the same of x's transpose, from the same read of x.
    """
    import torch
    rows, cols, ld = _matrix(x, "x")
    if dtype is None:
        dtype = torch.float8_e4m3fn
    kind = _torch_types().get(dtype)
    if kind not in (2, 3):
        raise TypeError(f"unsupported 8-bit dtype {dtype}")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    dev = x.device

    def outputs(r, c):
        pitch = -(-c // 16) * 16
        return (torch.empty_strided((r, c), (pitch, 1), dtype=dtype, device=dev),
                torch.empty((-(-c // 128), -(-r // block_rows)), dtype=torch.float32, device=dev))

    q, scale = outputs(rows, cols)
    args = QuantizeArgs(x=x.data_ptr(), q=q.data_ptr(), scale=scale.data_ptr(),
                        x_dtype=_type(x, "x", (0, 1)), q_dtype=kind, block_rows=block_rows,
                        rows=rows, cols=cols, ld_x=ld, ld_q=q.stride(0), ld_scale=scale.shape[1])
    out = (q, scale)
    if transposed:
        qt, scale_t = outputs(cols, rows)
        args.qt, args.scale_t = qt.data_ptr(), scale_t.data_ptr()
        args.ld_qt, args.ld_scale_t = qt.stride(0), scale_t.shape[1]
        out = (q, scale, qt, scale_t)
    _run(tr_quantize_fp8, args, dev)
    return out


def _block_rows(scale, rows, k, name, device):
    """Rows to a scale, told by the scales' shape."""
    kb, rb, ld = _matrix(scale, name, device)
    if _type(scale, name, (0,)) != 0 or kb != -(-k // 128) or rb not in (rows, -(-rows // 128)):
        raise ValueError(f"{name} has shape {tuple(scale.shape)}, expected "
                         f"[{-(-k // 128)}, {rows} or {-(-rows // 128)}]")
    return (1 if rb == rows else 128), ld


@_on_stream
def matmul_fp8(a, scale_a, b, scale_b, *, out=None, out_dtype=None, accumulate=False):
    """Product ``a @ b.T`` of two 8-bit operands [m, k] and [n, k] with their scales.

    The operands are as ``quantize_fp8`` returns them (or its transposed pair):
    scales of shape [ceil(k/128), rows] hold one for each 1 x 128 values, of
    shape [ceil(k/128), ceil(rows/128)] one for each 128 x 128.  The output is
    ``out`` (fp32 or bf16, may be a strided view) or a new matrix of
    ``out_dtype`` (bf16 by default); ``accumulate`` adds to ``out``.
    """
    import torch
    m, k, lda = _matrix(a, "a")
    dev = a.device
    n, kb, ldb = _matrix(b, "b", dev)
    if kb != k:
        raise ValueError(f"a and b contract over {k} and {kb} values")
    a_rows, ld_sa = _block_rows(scale_a, m, k, "scale_a", dev)
    b_rows, ld_sb = _block_rows(scale_b, n, k, "scale_b", dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an output to add to")
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out_dtype is not out's dtype")
    om, on, ld_out = _matrix(out, "out", dev)
    if (om, on) != (m, n):
        raise ValueError(f"out has shape {(om, on)}, expected {(m, n)}")
    args = MatmulFp8Args(a.data_ptr(), scale_a.data_ptr(), b.data_ptr(), scale_b.data_ptr(),
                         out.data_ptr(), _type(a, "a", (2, 3)), _type(b, "b", (2, 3)),
                         _type(out, "out", (0, 1)), a_rows, b_rows, int(bool(accumulate)), m, n, k,
                         lda, ldb, ld_out, ld_sa, ld_sb)
    _run(tr_matmul_fp8, args, dev)
    return out


@_on_stream
def layernorm(x, gamma, beta=None, *, eps=1e-5, out=None):
    """Layer norm over the rows of a CUDA matrix (fp32 or bf16).

    Returns ``(y, mean, rstd)``: y of x's type (``out`` if given), the rows'
    means and reciprocal deviations in fp32 for ``layernorm_backward``.
    ``gamma`` and ``beta`` are fp32 or bf16, both the same.
    """
    import torch
    rows, cols, ld = _matrix(x, "x")
    dev = x.device
    _vector(gamma, "gamma", cols, dev)
    if beta is not None:
        _vector(beta, "beta", cols, dev)
        if beta.dtype != gamma.dtype:
            raise TypeError("gamma and beta must have the same dtype")
    if out is None:
        out = torch.empty((rows, cols), dtype=x.dtype, device=dev)
    if _matrix(out, "out", dev)[:2] != (rows, cols) or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    stats = torch.empty((2, rows), dtype=torch.float32, device=dev)
    mean, rstd = stats[0], stats[1]
    args = LayernormArgs(x.data_ptr(), gamma.data_ptr(), None if beta is None else beta.data_ptr(),
                         out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _type(x, "x", (0, 1)),
                         _type(gamma, "gamma", (0, 1)), rows, cols, ld, _matrix(out, "out")[2], eps)
    _run(tr_layernorm, args, dev)
    return out, mean, rstd


@_on_stream
def layernorm_backward(dy, x, gamma, mean, rstd, *, bias=True, out=None):
    """Gradients of ``layernorm``: ``(dx, dgamma, dbeta)``, dx of x's type (``out``
    if given), the others in fp32; without ``bias`` dbeta is None."""
    import torch
    rows, cols, ld = _matrix(x, "x")
    dev = x.device
    r, c, ld_dy = _matrix(dy, "dy", dev)
    if (r, c) != (rows, cols) or dy.dtype != x.dtype:
        raise ValueError("dy must match x in shape and dtype")
    _vector(gamma, "gamma", cols, dev)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _vector(t, name, rows, dev)
        _type(t, name, (0,))
    if out is None:
        out = torch.empty((rows, cols), dtype=x.dtype, device=dev)
    r, c, ld_dx = _matrix(out, "out", dev)
    if (r, c) != (rows, cols) or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    dgamma = torch.empty(cols, dtype=torch.float32, device=dev)
    dbeta = torch.empty(cols, dtype=torch.float32, device=dev) if bias else None
    size = tr_layernorm_backward_workspace(rows, cols)
    workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    args = LayernormBackwardArgs(dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), mean.data_ptr(),
                                 rstd.data_ptr(), out.data_ptr(), dgamma.data_ptr(),
                                 dbeta.data_ptr() if bias else None, workspace.data_ptr(), size,
                                 _type(x, "x", (0, 1)), _type(gamma, "gamma", (0, 1)), rows, cols,
                                 ld_dy, ld, ld_dx)
    _run(tr_layernorm_backward, args, dev)
    return out, dgamma, dbeta
