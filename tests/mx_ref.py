"""Plain implementation of the microscaled operators in 64 bits (numpy, CPU),
from the definitions of the OCP Microscaling Formats (MX) Specification v1.0.
It shares nothing with the library: elements are found by search among all
values of the type, codes are decoded bit by bit, and scales are addressed by
the formula of the storage layout."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 32
FORMATS = ("mxfp8", "mxfp4")
EMAX = {"mxfp8": 8, "mxfp4": 2}
# half a step of the 16-bit outputs, relative, and half the smallest subnormal
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def magnitudes(fmt: str) -> np.ndarray:
    """The non-negative finite values by code: E4M3 (0..0x7E), E2M1 (0..7)."""
    if fmt == "mxfp8":
        e, m, bias, codes = 4, 3, 7, 127
    else:
        e, m, bias, codes = 2, 1, 1, 8
    out = []
    for c in range(codes):
        ex, man = c >> m, c & ((1 << m) - 1)
        out.append(man * 2.0 ** (1 - bias - m) if ex == 0
                   else (2 ** m + man) * 2.0 ** (ex - bias - m))
    return np.array(out)


def nearest_codes(y: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of the elements nearest to |y|, ties to the even code, saturating."""
    v = magnitudes(fmt)
    hi = np.clip(np.searchsorted(v, y, side="left"), 1, len(v) - 1)
    lo = hi - 1
    dl, dh = y - v[lo], v[hi] - y
    pick_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(pick_hi, hi, lo)


def quantize(x: np.ndarray, fmt: str):
    """(codes with the sign in the top bit, scale bytes) of the rows of x."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    full = np.zeros((rows, nb * BLOCK))
    full[:, :cols] = x
    full = full.reshape(rows, nb, BLOCK)
    bad = ~np.isfinite(full).all(2)
    safe = np.where(bad[..., None], 0.0, full)
    amax = np.abs(safe).max(2)
    _, e = np.frexp(amax)  # amax = f 2^e, f in [1/2, 1)
    exp = np.where(amax > 0, np.clip(e - 1 - EMAX[fmt], -127, 127), -127)
    y = np.abs(safe) / np.exp2(exp.astype(np.float64))[..., None]
    codes = nearest_codes(y, fmt)
    sign = 128 if fmt == "mxfp8" else 8
    codes = np.where(bad[..., None], 0, codes + sign * np.signbit(safe))
    scales = np.where(bad, 255, exp + 127)
    return codes.reshape(rows, nb * BLOCK)[:, :cols].astype(np.uint8), scales.astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray, fmt: str) -> np.ndarray:
    """What codes (rows, cols) and scale bytes (rows, blocks) stand for."""
    sign = 128 if fmt == "mxfp8" else 8
    mag = codes & (sign - 1)
    v = np.append(magnitudes(fmt), np.nan) if fmt == "mxfp8" else magnitudes(fmt)
    v = np.where(codes >= sign, -v[mag], v[mag])
    x = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(x, BLOCK, 1)[:, :codes.shape[1]]


def row_bytes(cols: int, fmt: str) -> int:
    return cols if fmt == "mxfp8" else (cols + 1) // 2


def pack(codes: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "mxfp8":
        return codes
    rows, cols = codes.shape
    even = np.zeros((rows, (cols + 1) // 2 * 2), np.uint8)
    even[:, :cols] = codes
    return even[:, 0::2] | even[:, 1::2] << 4


def unpack(data: np.ndarray, cols: int, fmt: str) -> np.ndarray:
    if fmt == "mxfp8":
        return data[:, :cols]
    both = np.stack((data & 15, data >> 4), 2).reshape(data.shape[0], -1)
    return both[:, :cols]


def scale_places(rows: int, cols: int) -> np.ndarray:
    """Byte index of the scale of (row, block)."""
    tiles = -(-cols // 128)
    r = np.arange(rows)[:, None]
    b = np.arange(-(-cols // BLOCK))[None, :]
    return ((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4


def tile_scales(scales: np.ndarray, cols: int) -> np.ndarray:
    rows = scales.shape[0]
    out = np.zeros(-(-rows // 128) * -(-cols // 128) * 512, np.uint8)
    out[scale_places(rows, cols)] = scales
    return out


def act(x: np.ndarray, name: str) -> np.ndarray:
    if name == "relu":
        return np.where(x > 0, x, 0.0)
    if name == "gelu":
        t = torch.from_numpy(np.ascontiguousarray(x))
        return (t * torch.special.ndtr(t)).numpy()
    return x


def product(a: np.ndarray, b: np.ndarray, bias, name: str):
    """(act(a @ b.T + bias), bound on the fp32 sum's error before rounding).

    The products are exact (4 + 4 significant bits).  An MMA adds 32 or more of
    them to the accumulator; each addition, within it or of its result, is off
    by at most 2^-23 of the largest magnitude in play, itself at most
    S = sum |a b| + |bias|.  Counting one for every 16 products and 16 more for
    joining the parts of K, the bias and the activation's own error
    (GELU: derivative at most 1.13, |error| <= 2e-7 |x|)."""
    x = a @ b.T
    s = np.abs(a) @ np.abs(b).T
    if bias is not None:
        x = x + bias
        s = s + np.abs(bias)
    k = a.shape[1]
    return act(x, name), 1.13 * (math.ceil(k / 16) + 16) * 2.0 ** -23 * s


def norm(x: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    with np.errstate(invalid="ignore", divide="ignore"):
        return x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * w


def to_np(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def round_to(x: np.ndarray, dtype) -> np.ndarray:
    """x (64 bits) rounded once to a 16-bit type, as 64-bit values."""
    with np.errstate(over="ignore", invalid="ignore"):
        if dtype == torch.float16:
            return x.astype(np.float16).astype(np.float64)
        # bf16: round the fp64 value at 8 significant bits, ties to even
        m, e = np.frexp(x)
        step = np.exp2(np.maximum(e - 8, -133).astype(np.float64))
        y = np.round(x / step) * step
        return np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, x), np.where(np.isfinite(x), y, x))
