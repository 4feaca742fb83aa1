"""Python binding of libttcmx (argument marshalling only): microscaled (MX)
operands for the products of a linear layer.

As in ``ops``, every function forwards device pointers, sizes, strides and the
current CUDA stream of PyTorch to a C ABI (``include/gemm_mx.h``), whose CUDA
kernels do all arithmetic; there is no fallback.  Checks of tensors and
allocation of outputs are in a small CPython extension (``csrc/mx_bind.cpp``),
since a call's kernels may take only a few microseconds.

    q = mx_quantize(w, "mxfp4")                  # weight (N, K), once
    y, h = rms_norm(x, g, residual=r, format="mxfp4")
    c = gemm_mx(y, q, bias, "gelu")              # GELU(norm(x + r) @ w.T + bias)

Formats are those of the OCP Microscaling Formats (MX) Specification v1.0:
"mxfp8" (E4M3 elements) and "mxfp4" (E2M1), one power-of-two scale for each 32
elements of a row.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import build, ops

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libttcmx.so")

FORMATS = {"mxfp8": 1, "mxfp4": 2}
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
BLOCK = 32

_lib = None
_bind = None

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
    global _lib, _bind
    if _lib is None:
        bind_path = build.bind_path()
        for path in (LIB_PATH, bind_path):
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with "
                    "`python -m tiled_tensor_core_05_b200.build` (there is no CPU fallback)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        spec = importlib.util.spec_from_file_location("_mxbind", bind_path)
        bind = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(bind)
        bind.bind(*(ctypes.cast(getattr(handle, name), _p).value for name in
                    ("mx_quantize", "mx_dequantize", "mx_rms_norm", "mx_gemm")))
        _bind, _lib = bind, handle
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


def _mx(q: MxTensor, what: str) -> torch.device:
    """Checks an MX input; its device."""
    if not isinstance(q, MxTensor):
        raise TypeError(f"{what} must be an MxTensor")
    if not q.data.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device")
    return q.data.device


def _mx_out(q: MxTensor, x: torch.Tensor, format: str) -> None:
    """Checks an MX output for the matrix x."""
    if _mx(q, "out") != x.device or q.shape != tuple(x.shape) or q.format != format:
        raise ValueError(f"out must be {tuple(x.shape)} {format} on {x.device}, got {q!r}")


def _new_type(dtype: torch.dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.float16 or torch.bfloat16")
    return _DTYPES[dtype]


def _made(data: torch.Tensor, scales: torch.Tensor, ld: int, rows: int, cols: int,
          format: str) -> MxTensor:
    """An MxTensor of outputs the binding has allocated: right by construction."""
    q = object.__new__(MxTensor)
    q.data, q.scales, q.ld, q.rows, q.cols, q.format = data, scales, ld, rows, cols, format
    return q


def _handle(stream):
    """None (the device's current stream) or the raw handle of a stream."""
    return stream if stream is None else ops._stream_handle(stream, None)


def _loaded():
    """The binding, with the library loaded."""
    if _bind is None:
        mx_lib()
    return _bind


def mx_quantize(x: torch.Tensor, format: str, out: MxTensor | None = None, *,
                stream=None) -> MxTensor:
    """The MX form of the rows of ``x`` (fp16 or bf16, CUDA, contiguous columns,
    rows 16-byte aligned).  Exact: every element is the correctly rounded
    quotient by its block's scale.  Asynchronous on ``stream`` (default: the
    current stream)."""
    fmt = _format(format)
    bind = _bind or _loaded()
    if out is None:
        rc, data, scales, ld = bind.quantize(x, fmt, None, None, None, _handle(stream))
        out = _made(data, scales, ld, *x.shape, format)
    else:
        _mx_out(out, x, format)
        rc = bind.quantize(x, fmt, out.data, out.scales, out.ld, _handle(stream))[0]
    if rc:
        ops._check(rc, "mx_quantize")
    return out


def mx_dequantize(q: MxTensor, dtype: torch.dtype = torch.float16,
                  out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """The values ``q`` stands for, rounded to ``dtype`` (fp16 or bf16; of
    ``out`` when given)."""
    _mx(q, "q")
    rc, out = (_bind or _loaded()).dequantize(
        q.data, q.scales, q.rows, q.cols, q.ld, FORMATS[q.format], out,
        _new_type(dtype) if out is None else None, _handle(stream))
    if rc:
        ops._check(rc, "mx_dequantize")
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
    bind = _bind or _loaded()
    if format is None:
        rc, y, _, _, h = bind.rms_norm(x, weight, eps, residual, residual_out, 0, out, None, None,
                                       _handle(stream))
    elif out is None:
        rc, data, scales, ld, h = bind.rms_norm(x, weight, eps, residual, residual_out,
                                                _format(format), None, None, None,
                                                _handle(stream))
        y = _made(data, scales, ld, *x.shape, format)
    else:
        _mx_out(out, x, format)
        rc, _, _, _, h = bind.rms_norm(x, weight, eps, residual, residual_out, _format(format),
                                       out.data, out.scales, out.ld, _handle(stream))
        y = out
    if rc:
        ops._check(rc, "mx_rms_norm")
    if residual is None:
        return y
    return y, h if residual_out is None else residual_out


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
    act = ops._ACTS[act] if isinstance(act, str) else int(act)
    rc, c = (_bind or _loaded()).gemm(
        a.data, a.scales, b.data, b.scales, a.rows, b.rows, a.cols, a.ld, b.ld,
        FORMATS[a.format], bias, act, out, _new_type(dtype) if out is None else None,
        _handle(stream))
    if rc:
        ops._check(rc, "mx_gemm")
    return c if out is None else out


def mx_device_status(stream=None, device=None) -> int:
    """Synchronise and return (then clear) libttcmx's device status word (0 = ok)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    st = ctypes.c_int(0)
    with torch.cuda.device(dev):
        ops._check(mx_lib().mx_get_device_status(ops._stream_handle(stream, dev),
                                                 ctypes.byref(st)), "mx_get_device_status")
    return int(st.value)
