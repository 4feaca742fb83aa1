"""Plain implementation of the feed-forward operators in 64 bits (torch, CPU), with
bounds on what fp32 sums and 16-bit roundings may be off by.  It shares nothing with
the library: 4-bit words are decoded bit by bit by the formula of the layout."""
from __future__ import annotations

import math

import torch

ACTS = ("silu", "gelu", "relu", "none")
# half a step of the 16-bit types, relative, and half the smallest subnormal
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
STEEPEST = 1.13  # |act'| is at most 1.0998 (SiLU), 1.129 (GELU), 1
BEND = 0.8       # |act''| is at most 0.5 (SiLU), 2 phi(0) = 0.798 (GELU)


def normal_cdf(x):
    """Right in relative terms down the negative tail, too (1 + erf cancels there)."""
    return 0.5 * torch.special.erfc(x * -math.sqrt(0.5))


def act(x, name):
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return x * normal_cdf(x)
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    return x


def slope(x, name):
    if name == "silu":
        p = torch.sigmoid(x)
        return p * (1 + x * (1 - p))
    if name == "gelu":
        return normal_cdf(x) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return (x > 0).double()
    return torch.ones_like(x)


def sum_bound(k, magnitudes):
    """What an fp32 sum of k products may be off by.  An MMA adds 16 of them to the accumulator;
    each addition, within it or of its result, is off by at most 2^-23 of the largest magnitude in
    play, itself at most the sum of magnitudes.  Counting one for every 16 products and 16 more for
    joining the parts of K and the scales of groups (of 32 columns or more)."""
    return (math.ceil(k / 16) + 16) * 2.0 ** -23 * magnitudes


def act_error(x, name):
    """What the activation's fp32 evaluation may be off by, relative to its value: 2^-18 + x^2 2^-22
    for GELU; SiLU's exponential and reciprocal are right to a few 2^-22 and its exponent's rounding
    adds |x| 2^-23; nothing for the others."""
    if name == "gelu":
        return 2.0 ** -18 + x * x * 2.0 ** -22
    if name == "silu":
        return 2.0 ** -20 + x.abs() * 2.0 ** -22
    return torch.zeros_like(x)


class Gated:
    """h = act(x wg^T) * (x wu^T) and its gradients, all fp64 CPU tensors."""

    def __init__(self, x, wg, wu, name):
        self.x, self.wg, self.wu, self.name = x, wg, wu, name
        self.g, self.u = x @ wg.t(), x @ wu.t()
        k = x.shape[1]
        self.off_g = sum_bound(k, x.abs() @ wg.abs().t())
        self.off_u = sum_bound(k, x.abs() @ wu.abs().t())
        self.a = act(self.g, name)
        self.off_a = STEEPEST * self.off_g + act_error(self.g, name) * self.a.abs()
        self.h = self.a * self.u

    def h_bound(self, dtype):
        off = self.off_a * (self.u.abs() + self.off_u) + self.a.abs() * self.off_u
        off = off + 2.0 ** -23 * self.h.abs()
        return off * (1 + HALF[dtype]) + HALF[dtype] * self.h.abs() + TINY[dtype]

    def backward(self, dh, dtype):
        """{name: (value, bound)} of dx, dw_gate, dw_up."""
        r, tiny = HALF[dtype], TINY[dtype]
        s = slope(self.g, self.name)
        dg, du = dh * self.u * s, dh * self.a
        # the slope's error: its argument's, and its evaluation's (of values up to 1.13, with
        # GELU's x phi(x) and SiLU's x p (1 - p) below 0.3)
        off_s = BEND * self.off_g + 2.0 ** -18 + torch.where(
            self.g.abs() <= self.off_g, 1.0, 0.0) * (self.name == "relu")
        off_dg = dh.abs() * (self.u.abs() * off_s + self.off_u * (s.abs() + off_s))
        off_du = dh.abs() * self.off_a
        off_dg = off_dg * (1 + r) + (r + 2.0 ** -22) * dg.abs() + tiny
        off_du = off_du * (1 + r) + (r + 2.0 ** -22) * du.abs() + tiny
        self.dg, self.du = dg, du
        out = {}

        def product(name, k, value, magnitudes, off):
            out[name] = (value, (off + sum_bound(k, magnitudes + off)) * (1 + r) +
                         r * value.abs() + tiny)

        F, M = self.wg.shape[0], self.x.shape[0]
        product("dx", 2 * F, dg @ self.wg + du @ self.wu,
                dg.abs() @ self.wg.abs() + du.abs() @ self.wu.abs(),
                off_dg @ self.wg.abs() + off_du @ self.wu.abs())
        product("dw_gate", M, dg.t() @ self.x, dg.abs().t() @ self.x.abs(),
                off_dg.t() @ self.x.abs())
        product("dw_up", M, du.t() @ self.x, du.abs().t() @ self.x.abs(),
                off_du.t() @ self.x.abs())
        return out


def close(got, want, bound, what=""):
    """got: a device tensor; want, bound: fp64 CPU."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; first {at}: "
                             f"got {got[at].item()}, want {want[at].item()}, "
                             f"bound {bound[at].item()}")


def rounded(x, dtype):
    """fp64 values rounded once to a 16-bit type (x has at most 24 significant bits)."""
    return x.float().to(dtype)


# ------------------------------------------------------------------- 4-bit weights ---


def pack_words(codes, fill=0):
    """(rows, cols) codes -> the data bytes, word by word; columns that do not exist hold `fill`."""
    rows, cols = codes.shape
    words = (cols + 7) // 8
    full = torch.full((rows, words * 8), fill, dtype=torch.int64)
    full[:, :cols] = codes
    out = torch.zeros((rows, words * 4), dtype=torch.uint8)
    for w in range(words):
        v = torch.zeros(rows, dtype=torch.int64)
        for j in range(8):
            v |= full[:, 8 * w + j] << (4 * (j // 2) + 16 * (j % 2))
        for b in range(4):
            out[:, 4 * w + b] = ((v >> (8 * b)) & 255).to(torch.uint8)
    return out


def weight(codes, scales, zeros, group):
    """codes (rows, cols), scales and zeros (or None) (groups, rows) -> fp64 (rows, cols)."""
    rows, cols = codes.shape
    k = torch.arange(cols) // group
    z = torch.full(scales.shape, 8.0, dtype=torch.float64) if zeros is None else zeros.double()
    return (codes.double() - z.t()[:, k]) * scales.double().t()[:, k]


def w4_bound(x, w, bias, name, dtype):
    """(value, bound) of act(x w^T + bias)."""
    v, m = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        v, m = v + bias, m + bias.abs()
    off = sum_bound(x.shape[1], m)
    y = act(v, name)
    off = STEEPEST * off + act_error(v, name) * y.abs()
    return y, off * (1 + HALF[dtype]) + HALF[dtype] * y.abs() + TINY[dtype]
