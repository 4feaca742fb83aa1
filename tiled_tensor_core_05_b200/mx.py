"""Python binding of libttcmx (argument marshalling only): microscaled (MX)
operands for the products of a linear layer.

As in ``ops``, every function forwards device pointers, sizes, strides and the
current CUDA stream of PyTorch to a C ABI (``include/gemm_mx.h``), whose CUDA
kernels do all arithmetic; there is no fallback.

    q = mx_quantize(w, "mxfp4")                  # weight (N, K), once
    y, h = rms_norm(x, g, residual=r, format="mxfp4")
    c = gemm_mx(y, q, bias, "gelu")              # GELU(norm(x + r) @ w.T + bias)

Formats are those of the OCP Microscaling Formats (MX) Specification v1.0:
"mxfp8" (E4M3 elements) and "mxfp4" (E2M1), one power-of-two scale for each 32
elements of a row.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import ops

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libttcmx.so")

FORMATS = {"mxfp8": 1, "mxfp4": 2}
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
BLOCK = 32

_lib = None

_p, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_SIGNATURES = {
    "mx_row_bytes": ([_i64, _int], _i64),
    "mx_scale_bytes": ([_i64, _i64], _i64),
    "mx_quantize": ([_p] * 3 + [_i64] * 4 + [_int] * 2 + [_p], _int),
    "mx_dequantize": ([_p] * 3 + [_i64] * 4 + [_int] * 2 + [_p], _int),
    "mx_rms_norm": ([_p] * 6 + [_i64] * 6 + [ctypes.c_float] + [_int] * 2 + [_p], _int),
    "mx_gemm": ([_p] * 6 + [_i64] * 6 + [_int] * 3 + [_p], _int),
    "mx_get_device_status": ([_p, ctypes.POINTER(_int)], _int),
    "mx_abi_version": ([], _int),
}


def mx_lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m tiled_tensor_core_05_b200.build` (there is no CPU fallback)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def _format(fmt: str) -> int:
    if fmt not in FORMATS:
        raise ValueError(f"format must be one of {sorted(FORMATS)}, got {fmt!r}")
    return FORMATS[fmt]


def _round(n: int, to: int) -> int:
    return -(-n // to) * to


def mx_row_bytes(cols: int, format: str) -> int:
    """Bytes of a row of ``cols`` elements."""
    if format == "mxfp8":
        return cols
    _format(format)
    return (cols + 1) // 2


def mx_scale_bytes(rows: int, cols: int) -> int:
    """Bytes of the scales of a (rows, cols) matrix."""
    return -(-rows // 128) * -(-cols // 128) * 512


class MxTensor:
    """A (rows, cols) MX matrix: ``data`` uint8 (rows, bytes), rows a multiple
    of 16 bytes apart, and ``scales`` uint8, flat, in 128 x 4 tiles
    (``mx_tile_scales``)."""

    __slots__ = ("data", "scales", "rows", "cols", "format", "ld")

    def __init__(self, data: torch.Tensor, scales: torch.Tensor, rows: int, cols: int,
                 format: str):
        need = mx_row_bytes(cols, format)
        if data.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
            raise TypeError("data and scales must be torch.uint8")
        shape = data.shape
        if len(shape) != 2 or shape[0] != rows or shape[1] < need:
            raise ValueError(f"data must be ({rows}, >= {need}), got {tuple(shape)}")
        step, unit = data.stride()
        if unit != 1 and shape[1] > 1:
            raise ValueError("the bytes of a row must be contiguous")
        if scales.dim() != 1 or not scales.is_contiguous() or \
                scales.numel() < mx_scale_bytes(rows, cols):
            raise ValueError(f"scales must be flat, contiguous, >= {mx_scale_bytes(rows, cols)} "
                             "bytes")
        if data.device != scales.device:
            raise ValueError("data and scales must be on one device")
        self.data, self.scales = data, scales
        self.rows, self.cols, self.format = rows, cols, format
        # bytes between rows (a single row has no meaningful stride)
        self.ld = step if rows > 1 else (need + 15) // 16 * 16

    @property
    def shape(self) -> tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self) -> torch.device:
        return self.data.device

    def __repr__(self):
        return f"MxTensor({self.rows} x {self.cols}, {self.format}, {self.device})"


def mx_empty(rows: int, cols: int, format: str, device) -> MxTensor:
    """An uninitialised MX matrix."""
    q = object.__new__(MxTensor)  # right by construction: no checks
    q.ld = _round(mx_row_bytes(cols, format), 16)
    q.data = torch.empty((rows, q.ld), dtype=torch.uint8, device=device)
    q.scales = torch.empty((mx_scale_bytes(rows, cols),), dtype=torch.uint8, device=device)
    q.rows, q.cols, q.format = rows, cols, format
    return q


def mx_tile_scales(scales: torch.Tensor) -> torch.Tensor:
    """(rows, ceil(cols / 32)) E8M0 bytes, one row after the other -> the
    tiled layout of ``MxTensor.scales`` (places without a block are 0)."""
    rows, blocks = scales.shape
    r, b = -(-rows // 128), -(-blocks // 4)
    t = torch.zeros((r * 128, b * 4), dtype=torch.uint8, device=scales.device)
    t[:rows, :blocks] = scales
    return t.view(r, 4, 32, b, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def mx_untile_scales(scales: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """The reverse of :func:`mx_tile_scales`: (rows, ceil(cols / 32)) bytes."""
    r, b = -(-rows // 128), -(-cols // 128)
    t = scales[:r * b * 512].view(r, b, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, b * 4)
    return t[:rows, :-(-cols // BLOCK)]


def _dtype(t: torch.Tensor, what: str) -> int:
    """The code of the 16-bit type of the CUDA tensor ``t``."""
    code = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        raise TypeError(f"{what} must be a torch.float16 or torch.bfloat16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return code


def _matrix(t: torch.Tensor, what: str, shape, dtype, device) -> int:
    """Checks a matrix; its row stride in elements (of a single row, whose
    stride means nothing, the columns rounded up to 8)."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.shape != shape or len(shape) != 2:
        raise ValueError(f"{what} must be a matrix {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")
    step, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError(f"the columns of {what} must be contiguous (stride(1) == 1)")
    return step if shape[0] > 1 else (shape[1] + 7) // 8 * 8


def _vector(t: torch.Tensor, what: str, n: int, dtype, device) -> int:
    """Checks a vector; its address."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what} must be {n} contiguous values on {device}")
    return t.data_ptr()


def _mx(q: MxTensor, what: str) -> torch.device:
    """Checks an MX input; its device."""
    if not isinstance(q, MxTensor):
        raise TypeError(f"{what} must be an MxTensor")
    if not q.data.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device")
    return q.data.device


def _mx_out(q: MxTensor, rows: int, cols: int, format: str, device) -> None:
    if _mx(q, "out") != device or q.rows != rows or q.cols != cols or q.format != format:
        raise ValueError(f"out must be ({rows}, {cols}) {format} on {device}, got {q!r}")


def _new(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """A new matrix whose rows start on 16 bytes."""
    if cols % 8 == 0:
        return torch.empty((rows, cols), dtype=dtype, device=device)
    return torch.empty((rows, _round(cols, 8)), dtype=dtype, device=device)[:, :cols]


def _alloc(stream, device, make, *args):
    """make(*args) with the memory belonging to the stream that will write it."""
    if stream is None:
        return make(*args)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return make(*args)


def _call(name: str, device: torch.device, stream, *args) -> None:
    """The library call, with ``device`` current, on ``stream`` or the device's
    current stream."""
    if torch._C._cuda_getDevice() != device.index:
        with torch.cuda.device(device):
            return _call(name, device, stream, *args)
    handle = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else \
        ops._stream_handle(stream, device)
    rc = getattr(_lib or mx_lib(), name)(*args, handle)
    if rc:
        ops._check(rc, name)


def mx_quantize(x: torch.Tensor, format: str, out: MxTensor | None = None, *,
                stream=None) -> MxTensor:
    """The MX form of the rows of ``x`` (fp16 or bf16, CUDA, contiguous columns,
    rows 16-byte aligned).  Exact: every element is the correctly rounded
    quotient by its block's scale.  Asynchronous on ``stream`` (default: the
    current stream)."""
    fmt = _format(format)
    dtype, dev, shape = _dtype(x, "x"), x.device, x.shape
    ldx = _matrix(x, "x", shape, x.dtype, dev)
    rows, cols = shape
    if out is None:
        out = _alloc(stream, dev, mx_empty, rows, cols, format, dev)
    else:
        _mx_out(out, rows, cols, format, dev)
    _call("mx_quantize", dev, stream, x.data_ptr(), out.data.data_ptr(), out.scales.data_ptr(),
          rows, cols, ldx, out.ld, dtype, fmt)
    return out


def mx_dequantize(q: MxTensor, dtype: torch.dtype = torch.float16,
                  out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """The values ``q`` stands for, rounded to ``dtype`` (fp16 or bf16; of
    ``out`` when given)."""
    dev = _mx(q, "q")
    if out is None:
        if dtype not in _DTYPES:
            raise TypeError("dtype must be torch.float16 or torch.bfloat16")
        out = _alloc(stream, dev, _new, q.rows, q.cols, dtype, dev)
    code = _dtype(out, "out")
    ldx = _matrix(out, "out", (q.rows, q.cols), out.dtype, dev)
    _call("mx_dequantize", dev, stream, q.data.data_ptr(), q.scales.data_ptr(), out.data_ptr(),
          q.rows, q.cols, q.ld, ldx, code, FORMATS[q.format])
    return out


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor | None = None, *, format: str | None = None, out=None,
             residual_out: torch.Tensor | None = None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the rows, with h = x or, with
    ``residual``, x + residual rounded to their type.

    Returns y, or (y, h) with a residual.  ``format`` None gives y in the type
    of ``x``; "mxfp8" / "mxfp4" an :class:`MxTensor` for :func:`gemm_mx`,
    quantised without rounding in between.  ``residual_out`` may be ``x`` or
    ``residual`` itself (updated in place)."""
    code, dtype, dev, shape = _dtype(x, "x"), x.dtype, x.device, x.shape
    ldx = _matrix(x, "x", shape, dtype, dev)
    rows, cols = shape
    fmt = 0 if format is None else _format(format)
    w = _vector(weight, "weight", cols, dtype, dev)
    h = r = None
    ldr = ldh = 0
    if residual is not None:
        ldr = _matrix(residual, "residual", shape, dtype, dev)
        r = residual.data_ptr()
        if residual_out is None:
            residual_out = _alloc(stream, dev, _new, rows, cols, dtype, dev)
        ldh = _matrix(residual_out, "residual_out", shape, dtype, dev)
        h = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if fmt:
        if out is None:
            out = _alloc(stream, dev, mx_empty, rows, cols, format, dev)
        else:
            _mx_out(out, rows, cols, format, dev)
        y, s, ldy = out.data.data_ptr(), out.scales.data_ptr(), out.ld
    else:
        if out is None:
            out = _alloc(stream, dev, _new, rows, cols, dtype, dev)
        ldy = _matrix(out, "out", shape, dtype, dev)
        y, s = out.data_ptr(), None
    _call("mx_rms_norm", dev, stream, x.data_ptr(), r, w, h, y, s, rows, cols, ldx, ldr, ldh, ldy,
          eps, code, fmt)
    return out if residual is None else (out, residual_out)


def gemm_mx(a: MxTensor, b: MxTensor, bias: torch.Tensor | None = None, act: str | int = "none",
            out: torch.Tensor | None = None, *, dtype: torch.dtype = torch.float16,
            stream=None) -> torch.Tensor:
    """C = act(A @ B.T + bias): ``a`` is (M, K), ``b`` (N, K), the layout of a
    linear layer's weight, both MX of one format; ``bias`` N values of the
    output's type or None; ``act`` "none" / "relu" / "gelu".  C is fp16 or
    bf16 (``dtype``, or the type of ``out``); the sums are fp32."""
    dev = _mx(a, "a")
    if _mx(b, "b") != dev or b.cols != a.cols or b.format != a.format:
        raise ValueError(f"a and b must share device, format and inner size: {a!r}, {b!r}")
    M, N, K = a.rows, b.rows, a.cols
    act = ops._ACTS[act] if isinstance(act, str) else int(act)
    if out is None:
        if dtype not in _DTYPES:
            raise TypeError("dtype must be torch.float16 or torch.bfloat16")
        out = _alloc(stream, dev, _new, M, N, dtype, dev)
    code = _dtype(out, "out")
    ldc = _matrix(out, "out", (M, N), out.dtype, dev)
    bias = None if bias is None else _vector(bias, "bias", N, out.dtype, dev)
    _call("mx_gemm", dev, stream, a.data.data_ptr(), a.scales.data_ptr(), b.data.data_ptr(),
          b.scales.data_ptr(), bias, out.data_ptr(), M, N, K, a.ld, b.ld, ldc, FORMATS[a.format],
          code, act)
    return out


def mx_device_status(stream=None, device=None) -> int:
    """Synchronise and return (then clear) libttcmx's device status word (0 = ok)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    st = ctypes.c_int(0)
    with torch.cuda.device(dev):
        ops._check(mx_lib().mx_get_device_status(ops._stream_handle(stream, dev),
                                                 ctypes.byref(st)), "mx_get_device_status")
    return int(st.value)
