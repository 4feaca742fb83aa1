"""Python binding of libttcff (argument marshalling only): the feed-forward part of
a model.

As in ``mx``, every function forwards device pointers, sizes, strides and the
current CUDA stream of PyTorch to a C ABI (``include/gemm_ff.h``), whose CUDA
kernels do all arithmetic; there is no fallback.  Checks of tensors and allocation
of outputs are in a CPython extension (``csrc/ff_bind.cpp``).

    h, gate, up = gemm_gated(x, w_gate, w_up, "silu", save=True)   # silu(x @ w_gate.T) * (x @ w_up.T)
    dx, dw_gate, dw_up = gemm_gated_backward(dh, x, w_gate, w_up, gate, up, "silu")

    w4 = w4_pack(codes, scales, zeros)       # 4 bits a weight, a scale for each group of columns
    y = gemm_w4(x, w4, bias, "gelu")         # gelu(x @ W.T + bias), few rows of x
    h = gemm_gated_w4(x, gate4, up4)         # the gated projections with such weights
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import build, ops

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libttcff.so")

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
GROUPS = (32, 64, 128)

_lib = None
_bind = None

_p, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_SIGNATURES = {
    "ff_gated": ([_p] * 6 + [_i64] * 9 + [_int] * 2 + [_p], _int),
    "ff_gated_backward": ([_p] * 11 + [_i64] * 14 + [_int] * 2 + [_p], _int),
    "ff_w4_gemm": ([_p] * 6 + [_i64] * 8 + [_int] * 3 + [_p], _int),
    "ff_w4_gated": ([_p] * 8 + [_i64] * 11 + [_int] * 3 + [_p], _int),
    "ff_get_device_status": ([_p, ctypes.POINTER(_int)], _int),
    "ff_abi_version": ([], _int),
}


def ff_lib() -> ctypes.CDLL:
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
        spec = importlib.util.spec_from_file_location("_ffbind", bind_path)
        bind = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(bind)
        bind.bind(*(ctypes.cast(getattr(handle, name), _p).value for name in
                    ("ff_gated", "ff_gated_backward", "ff_w4_gemm", "ff_w4_gated")))
        _bind, _lib = bind, handle
    return _lib


def _loaded():
    """The binding, with the library loaded."""
    if _bind is None:
        ff_lib()
    return _bind


def _act(act: str | int) -> int:
    if isinstance(act, str):
        if act not in ACTIVATIONS:
            raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
        return ACTIVATIONS[act]
    return int(act)


def _handle(stream):
    """None (the device's current stream) or the raw handle of a stream."""
    return stream if stream is None else ops._stream_handle(stream, None)


def gemm_gated(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: str | int = "silu",
               out: torch.Tensor | None = None, *, save: bool = False, stream=None):
    """h = act(x @ w_gate.T) * (x @ w_up.T): ``x`` (M, D), both weights (F, D), the layout of a
    linear layer's weight, fp16 or bf16; ``act`` "silu" / "gelu" / "relu" / "none".  Everything up
    to h's one rounding is fp32.

    Returns h (M, F) or, with ``save``, (h, gate, up): the two projections in fp32, which
    :func:`gemm_gated_backward` takes (rounded to 16 bits they would put the gradients 1.8 times
    as far from exact as a single rounding does; in fp32 it is 1.4 times).

    No autograd graph is recorded: the results of ``save`` are plain tensors, and a backward pass
    that reaches h without it, through inputs that require gradients, raises."""
    rc, h, gate, up = (_bind or _loaded()).gated(x, w_gate, w_up, _act(act), out, bool(save),
                                                 _handle(stream))
    if rc:
        ops._check(rc, "ff_gated")
    h = h if out is None else out
    return (h, gate, up) if save else h


def gemm_gated_backward(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor,
                        w_up: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                        act: str | int = "silu", *, need_x: bool = True, need_w: bool = True,
                        stream=None):
    """The gradients (dx, dw_gate, dw_up) of a loss from its gradient ``dh`` with respect to the h
    of ``gemm_gated(x, w_gate, w_up, act, save=True)`` and that call's ``gate`` and ``up``.
    Without ``need_x`` dx, without ``need_w`` both weights' are None and are not computed."""
    rc, *grads = (_bind or _loaded()).gated_backward(dh, x, w_gate, w_up, gate, up, _act(act),
                                                     bool(need_x), bool(need_w), _handle(stream))
    if rc:
        ops._check(rc, "ff_gated_backward")
    return tuple(grads)


class W4Tensor:
    """A (rows, cols) weight of 4-bit codes with a scale for each ``group`` (32, 64 or 128) columns
    of a row: W[n, k] = (code[n, k] - zeros[k // group, n]) * scales[k // group, n].

    ``data``    uint8 (rows, bytes), rows a multiple of 16 bytes apart; each 32-bit word holds 8
                consecutive columns, column 2 i of them in bits 4 i .. 4 i + 3 and column 2 i + 1 in
                bits 4 i + 16 .. 4 i + 19 (:func:`w4_pack` makes it);
    ``scales``  fp16 or bf16 (groups, rows), the type of the products' x;
    ``zeros``   uint8 (groups, rows), or None: 8 for all.
    Rows of scales and zeros start on 16 bytes, too.  A slice of rows (of multiples of 16) is a
    weight again: of data[a:b], scales[:, a:b], zeros[:, a:b]."""

    __slots__ = ("_rows", "_cols", "_group", "_args")

    def __init__(self, data: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None,
                 rows: int, cols: int, group: int):
        if group not in GROUPS:
            raise ValueError(f"group must be one of {GROUPS}, got {group!r}")
        if rows < 0 or cols < 0:
            raise ValueError(f"rows and cols must not be negative, got {rows}, {cols}")
        if data.dtype is not torch.uint8 or (zeros is not None and zeros.dtype is not torch.uint8):
            raise TypeError("data and zeros must be torch.uint8")
        if scales.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("scales must be torch.float16 or torch.bfloat16")
        need, groups = (cols + 7) // 8 * 4, -(-cols // group)
        shape = data.shape
        if len(shape) != 2 or shape[0] != rows or shape[1] < need:
            raise ValueError(f"data must be ({rows}, >= {need}), got {tuple(shape)}")
        strides = []
        for t, what, unit in ((data, "data", 16), (scales, "scales", 8), (zeros, "zeros", 16)):
            if t is None:
                strides.append(0)
                continue
            if t is not data and tuple(t.shape) != (groups, rows):
                raise ValueError(f"{what} must be ({groups}, {rows}), got {tuple(t.shape)}")
            if t.device != data.device:
                raise ValueError("data, scales and zeros must be on one device")
            step, one = t.stride()
            if one != 1 and t.shape[1] > 1:
                raise ValueError(f"the columns of {what} must be contiguous")
            if t.shape[0] <= 1 or t.numel() == 0:  # no meaningful stride
                step = -(-max(t.shape[1], 1) // unit) * unit
            elif step % unit:
                raise ValueError(f"the rows of {what} must start on 16 bytes")
            strides.append(step)
        self._rows, self._cols, self._group = rows, cols, group
        self._args = (data, scales, zeros, *strides)

    # (read-only: what the products take was checked together)
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    group = property(lambda self: self._group)
    data = property(lambda self: self._args[0])
    scales = property(lambda self: self._args[1])
    zeros = property(lambda self: self._args[2])

    @property
    def shape(self) -> tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self) -> torch.device:
        return self.data.device

    def __repr__(self):
        return (f"W4Tensor({self.rows} x {self.cols}, groups of {self.group}, "
                f"{'zeros' if self.zeros is not None else 'symmetric'}, {self.device})")


def _rows_on_16(t: torch.Tensor) -> torch.Tensor:
    """A copy of t whose rows start on 16 bytes."""
    unit = 16 // t.element_size()
    rows, cols = t.shape
    buf = torch.empty((rows, -(-cols // unit) * unit), dtype=t.dtype, device=t.device)
    buf[:, :cols] = t
    return buf[:, :cols]


def w4_pack(codes: torch.Tensor, scales: torch.Tensor,
            zeros: torch.Tensor | None = None, *, group: int = 128) -> W4Tensor:
    """The weight of ``codes`` (rows, cols) uint8 0 .. 15, ``scales`` (rows, groups) fp16 or bf16 and
    ``zeros`` (rows, groups) uint8 0 .. 15 or None (8 for all), on their device.  Done once, when a
    model is loaded; the weight keeps nothing of its arguments."""
    if codes.dtype is not torch.uint8 or codes.dim() != 2:
        raise TypeError("codes must be a matrix of torch.uint8")
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")
    rows, cols = codes.shape
    want = (rows, -(-cols // group))
    for t, what in ((scales, "scales"), (zeros, "zeros")):
        if t is not None and tuple(t.shape) != want:
            raise ValueError(f"{what} must be {want}, got {tuple(t.shape)}")
    for t, what in ((codes, "codes"), (zeros, "zeros")):
        if t is not None and t.numel() and int(t.max()) > 15:
            raise ValueError(f"{what} must be 0 .. 15")
    size = -(-cols // 32) * 32
    c = torch.nn.functional.pad(codes, (0, size - cols)).view(rows, size // 8, 8)
    even, odd = c[..., 0::2], c[..., 1::2]
    data = torch.cat([p[..., 0::2] | p[..., 1::2] << 4 for p in (even, odd)], 2)
    return W4Tensor(data.reshape(rows, size // 2), _rows_on_16(scales.t()),
                    None if zeros is None else _rows_on_16(zeros.t()), rows, cols, group)


def w4_unpack(w: W4Tensor) -> torch.Tensor:
    """The codes (rows, cols) of ``w``."""
    words = (w.cols + 7) // 8
    b = w.data[:, :words * 4].reshape(w.rows, words, 2, 2)  # word, parity, byte
    c = torch.stack((b & 15, b >> 4), 4)                    # ..., column pair of the byte
    return c.permute(0, 1, 3, 4, 2).reshape(w.rows, words * 8)[:, :w.cols]


def _check_w4(w: W4Tensor, what: str, x: torch.Tensor) -> None:
    if not isinstance(w, W4Tensor):
        raise TypeError(f"{what} must be a W4Tensor")
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    if x.dim() != 2 or x.shape[1] != w._cols:
        raise ValueError(f"x must be a matrix of {w.cols} columns, got {tuple(x.shape)}")


def gemm_w4(x: torch.Tensor, w: W4Tensor, bias: torch.Tensor | None = None,
            act: str | int = "none", out: torch.Tensor | None = None, *,
            stream=None) -> torch.Tensor:
    """y = act(x @ W.T + bias) for few rows of ``x`` (M, K), fp16 or bf16 as the scales of ``w``
    are; ``bias`` N values or None; ``act`` "none" / "relu" / "gelu" / "silu".  Codes and zero
    points are exact and sums are fp32: no weight is rounded.  The weight is read once for every
    64 rows.  There is no backward pass: one that reaches y raises."""
    _check_w4(w, "w", x)
    rc, y = (_bind or _loaded()).w4_gemm(x, *w._args, w._rows, w._group, bias, _act(act), out,
                                         _handle(stream))
    if rc:
        ops._check(rc, "ff_w4_gemm")
    return y if out is None else out


def gemm_gated_w4(x: torch.Tensor, w_gate: W4Tensor, w_up: W4Tensor, act: str | int = "silu",
                  out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """h = act(x @ Wg.T) * (x @ Wu.T) with two 4-bit weights of one shape and group, for few rows of
    ``x``: :func:`gemm_gated` in the form that serving takes."""
    _check_w4(w_gate, "w_gate", x)
    _check_w4(w_up, "w_up", x)
    if w_gate.shape != w_up.shape or w_gate.group != w_up.group or \
            (w_gate.zeros is None) != (w_up.zeros is None):
        raise ValueError(f"w_gate and w_up must share shape, group and zero points: {w_gate!r}, "
                         f"{w_up!r}")
    rc, h = (_bind or _loaded()).w4_gated(x, *w_gate._args, *w_up._args, w_gate._rows, w_gate._group,
                                          _act(act), out, _handle(stream))
    if rc:
        ops._check(rc, "ff_w4_gated")
    return h if out is None else out


def ff_device_status(stream=None, device=None) -> int:
    """Synchronise and return (then clear) libttcff's device status word (0 = ok)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    st = ctypes.c_int(0)
    with torch.cuda.device(dev):
        ops._check(ff_lib().ff_get_device_status(ops._stream_handle(stream, dev),
                                                 ctypes.byref(st)), "ff_get_device_status")
    return int(st.value)
