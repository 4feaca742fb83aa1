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

import contextlib
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
    _format(format)
    return cols if format == "mxfp8" else (cols + 1) // 2


def mx_scale_bytes(rows: int, cols: int) -> int:
    """Bytes of the scales of a (rows, cols) matrix."""
    return -(-rows // 128) * -(-cols // 128) * 512


class MxTensor:
    """A (rows, cols) MX matrix: ``data`` uint8 (rows, bytes), rows a multiple
    of 16 bytes apart, and ``scales`` uint8, flat, in 128 x 4 tiles
    (``mx_tile_scales``)."""

    __slots__ = ("data", "scales", "rows", "cols", "format")

    def __init__(self, data: torch.Tensor, scales: torch.Tensor, rows: int, cols: int,
                 format: str):
        need = mx_row_bytes(cols, format)
        if data.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("data and scales must be torch.uint8")
        if data.dim() != 2 or data.shape[0] != rows or data.shape[1] < need:
            raise ValueError(f"data must be ({rows}, >= {need}), got {tuple(data.shape)}")
        if data.shape[1] > 1 and data.stride(1) != 1:
            raise ValueError("the bytes of a row must be contiguous")
        if scales.dim() != 1 or not scales.is_contiguous() or \
                scales.numel() < mx_scale_bytes(rows, cols):
            raise ValueError(f"scales must be flat, contiguous, >= {mx_scale_bytes(rows, cols)} "
                             "bytes")
        if data.device != scales.device:
            raise ValueError("data and scales must be on one device")
        self.data, self.scales = data, scales
        self.rows, self.cols, self.format = int(rows), int(cols), format

    @property
    def shape(self) -> tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self) -> torch.device:
        return self.data.device

    def __repr__(self):
        return f"MxTensor({self.rows} x {self.cols}, {self.format}, {self.device})"

    def _ld(self) -> int:
        if self.rows > 1:
            return int(self.data.stride(0))
        return _round(mx_row_bytes(self.cols, self.format), 16)


def mx_empty(rows: int, cols: int, format: str, device) -> MxTensor:
    """An uninitialised MX matrix."""
    data = torch.empty((rows, _round(mx_row_bytes(cols, format), 16)), dtype=torch.uint8,
                       device=device)
    scales = torch.empty(mx_scale_bytes(rows, cols), dtype=torch.uint8, device=device)
    return MxTensor(data, scales, rows, cols, format)


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


def _matrix(t: torch.Tensor, what: str, shape=None, dtype=None, device=None) -> torch.Tensor:
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{what} must be {dtype or 'torch.float16 or torch.bfloat16'}")
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{what} must be a matrix{'' if shape is None else f' {tuple(shape)}'}, "
                         f"got {tuple(t.shape)}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{what} must be a CUDA tensor{'' if device is None else f' on {device}'}")
    return t


def _vector(t: torch.Tensor, what: str, n: int, dtype, device) -> torch.Tensor:
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what} must be {n} contiguous values on {device}")
    return t


def _mx(q: MxTensor, what: str, shape=None, format=None, device=None) -> MxTensor:
    if not isinstance(q, MxTensor):
        raise TypeError(f"{what} must be an MxTensor")
    if (shape is not None and q.shape != tuple(shape)) or \
            (format is not None and q.format != format):
        raise ValueError(f"{what} must be {shape} {format}, got {q!r}")
    if not q.data.is_cuda or (device is not None and q.device != device):
        raise ValueError(f"{what} must be on {device or 'a CUDA device'}")
    return q


def _owner(stream, device):
    """Context in which outputs are allocated: the stream that writes them."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _new(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """A new matrix whose rows start on 16 bytes."""
    return torch.empty((rows, _round(cols, 8)), dtype=dtype, device=device)[:, :cols]


def _call(name: str, device, stream, *args) -> None:
    with torch.cuda.device(device):
        ops._check(getattr(mx_lib(), name)(*args, ops._stream_handle(stream, device)), name)


def mx_quantize(x: torch.Tensor, format: str, out: MxTensor | None = None, *,
                stream=None) -> MxTensor:
    """The MX form of the rows of ``x`` (fp16 or bf16, CUDA, contiguous columns,
    rows 16-byte aligned).  Exact: every element is the correctly rounded
    quotient by its block's scale.  Asynchronous on ``stream`` (default: the
    current stream)."""
    fmt = _format(format)
    _matrix(x, "x")
    rows, cols = x.shape
    with _owner(stream, x.device):
        out = mx_empty(rows, cols, format, x.device) if out is None else \
            _mx(out, "out", (rows, cols), format, x.device)
    _call("mx_quantize", x.device, stream, x.data_ptr(), out.data.data_ptr(),
          out.scales.data_ptr(), rows, cols, ops._ld_padded(x), out._ld(), _DTYPES[x.dtype], fmt)
    return out


def mx_dequantize(q: MxTensor, dtype: torch.dtype = torch.float16,
                  out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """The values ``q`` stands for, rounded to ``dtype`` (fp16 or bf16; of
    ``out`` when given)."""
    _mx(q, "q")
    if out is None:
        if dtype not in _DTYPES:
            raise TypeError("dtype must be torch.float16 or torch.bfloat16")
        with _owner(stream, q.device):
            out = _new(q.rows, q.cols, dtype, q.device)
    _matrix(out, "out", q.shape, device=q.device)
    _call("mx_dequantize", q.device, stream, q.data.data_ptr(), q.scales.data_ptr(),
          out.data_ptr(), q.rows, q.cols, q._ld(), ops._ld_padded(out), _DTYPES[out.dtype],
          FORMATS[q.format])
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
    _matrix(x, "x")
    rows, cols = x.shape
    dev, dtype = x.device, x.dtype
    fmt = 0 if format is None else _format(format)
    _vector(weight, "weight", cols, dtype, dev)
    if residual is not None:
        _matrix(residual, "residual", (rows, cols), dtype, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    with _owner(stream, dev):
        if out is None:
            out = mx_empty(rows, cols, format, dev) if fmt else _new(rows, cols, dtype, dev)
        if residual is not None and residual_out is None:
            residual_out = _new(rows, cols, dtype, dev)
    h = residual_out
    if h is not None:
        _matrix(h, "residual_out", (rows, cols), dtype, dev)
    if fmt:
        _mx(out, "out", (rows, cols), format, dev)
        y, s, ldy = out.data.data_ptr(), out.scales.data_ptr(), out._ld()
    else:
        _matrix(out, "out", (rows, cols), dtype, dev)
        y, s, ldy = out.data_ptr(), None, ops._ld_padded(out)
    _call("mx_rms_norm", dev, stream, x.data_ptr(),
          None if residual is None else residual.data_ptr(), weight.data_ptr(),
          None if h is None else h.data_ptr(), y, s, rows, cols, ops._ld_padded(x),
          0 if residual is None else ops._ld_padded(residual),
          0 if h is None else ops._ld_padded(h), ldy, float(eps), _DTYPES[dtype], fmt)
    return out if residual is None else (out, h)


def gemm_mx(a: MxTensor, b: MxTensor, bias: torch.Tensor | None = None, act: str | int = "none",
            out: torch.Tensor | None = None, *, dtype: torch.dtype = torch.float16,
            stream=None) -> torch.Tensor:
    """C = act(A @ B.T + bias): ``a`` is (M, K), ``b`` (N, K), the layout of a
    linear layer's weight, both MX of one format; ``bias`` N values of the
    output's type or None; ``act`` "none" / "relu" / "gelu".  C is fp16 or
    bf16 (``dtype``, or the type of ``out``); the sums are fp32."""
    _mx(a, "a")
    M, K = a.shape
    _mx(b, "b", (b.rows, K) if isinstance(b, MxTensor) else None, a.format, a.device)
    N, dev = b.rows, a.device
    code = ops._ACTS[act] if isinstance(act, str) else int(act)
    if out is None:
        if dtype not in _DTYPES:
            raise TypeError("dtype must be torch.float16 or torch.bfloat16")
        with _owner(stream, dev):
            out = _new(M, N, dtype, dev)
    _matrix(out, "out", (M, N), device=dev)
    if bias is not None:
        _vector(bias, "bias", N, out.dtype, dev)
    _call("mx_gemm", dev, stream, a.data.data_ptr(), a.scales.data_ptr(), b.data.data_ptr(),
          b.scales.data_ptr(), None if bias is None else bias.data_ptr(), out.data_ptr(), M, N, K,
          a._ld(), b._ld(), ops._ld_padded(out), FORMATS[a.format], _DTYPES[out.dtype], code)
    return out


def mx_device_status(stream=None, device=None) -> int:
    """Synchronise and return (then clear) libttcmx's device status word (0 = ok)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    st = ctypes.c_int(0)
    with torch.cuda.device(dev):
        ops._check(mx_lib().mx_get_device_status(ops._stream_handle(stream, dev),
                                                 ctypes.byref(st)), "mx_get_device_status")
    return int(st.value)
