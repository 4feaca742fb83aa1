"""The microscaled operators on the GPU against the plain 64-bit implementation
of ``mx_ref``: quantisation and the norm's MX output bit by bit, products exactly
where the sums are exact and within a derived bound otherwise."""
import math

import numpy as np
import pytest
import torch

import mx_ref as ref
import tiled_tensor_core_05_b200 as ttc

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CANARY = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    ttc.mx_lib()
    yield
    torch.cuda.synchronize()
    assert ttc.mx_device_status() == 0


def dev16(x, dtype, pad_cols=0, pad_rows=0):
    """A device matrix of x's values with NaN around it."""
    rows, cols = x.shape
    buf = torch.full((rows + pad_rows, (cols + 7) // 8 * 8 + pad_cols), float("nan"), dtype=dtype,
                     device="cuda")
    buf[:rows, :cols] = torch.as_tensor(x).to(dtype).cuda()
    return buf[:rows, :cols]


def dev_vec(x, dtype):
    buf = torch.full(((x.size + 7) // 8 * 8 + 8,), float("nan"), dtype=dtype, device="cuda")
    buf[:x.size] = torch.as_tensor(x).to(dtype).cuda()
    return buf[:x.size]


class GuardedMx:
    """An MX output whose bytes outside the matrix hold a canary."""

    def __init__(self, rows, cols, fmt, pad=16):
        self.nb = ref.row_bytes(cols, fmt)
        self.buf = torch.full((rows + 2, (self.nb + 15) // 16 * 16 + pad), CANARY,
                              dtype=torch.uint8, device="cuda")
        self.sbuf = torch.full((ttc.mx_scale_bytes(rows, cols) + 64,), CANARY, dtype=torch.uint8,
                               device="cuda")
        self.rows, self.cols, self.fmt = rows, cols, fmt
        self.q = ttc.MxTensor(self.buf[1:rows + 1], self.sbuf[:-64], rows, cols, fmt)

    def check(self, codes, scales, what=""):
        got = self.buf.cpu().numpy()
        inside = got[1:self.rows + 1, :self.nb]
        want = ref.pack(codes, self.fmt)
        bad = np.argwhere(inside != want)
        assert not len(bad), f"{what}: {len(bad)} bytes differ, first {bad[0]}: " \
            f"{inside[tuple(bad[0])]} for {want[tuple(bad[0])]}"
        got[1:self.rows + 1, :self.nb] = CANARY
        assert (got == CANARY).all(), f"{what}: wrote outside the rows"
        s = self.sbuf.cpu().numpy()
        assert (s[-64:] == CANARY).all(), f"{what}: wrote behind the scales"
        assert np.array_equal(s[:-64], ref.tile_scales(scales, self.cols)), f"{what}: scales"


def host16(x, dtype):
    """x rounded to the type, as 64-bit values."""
    return torch.as_tensor(x).to(dtype).to(torch.float64).numpy()


def make_mx(codes, scales, fmt):
    """Device MxTensor of codes and scale bytes, with canaries in unused row bytes."""
    rows, cols = codes.shape
    g = GuardedMx(rows, cols, fmt)
    g.buf[1:rows + 1, :g.nb] = torch.from_numpy(ref.pack(codes, fmt).copy()).cuda()
    g.sbuf[:-64] = torch.from_numpy(ref.tile_scales(scales, cols)).cuda()
    return g.q


SIZES = [(1, 1), (1, 32), (2, 31), (3, 33), (7, 100), (33, 129), (128, 128), (129, 257),
         (200, 1000), (64, 4096), (5, 8199)]


# ------------------------------------------------------------------ quantisation ---


def spread_values(rng, rows, cols):
    """Values over many powers of two, with zeros, ties and whole zero blocks."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 8, (rows, 1)))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    ties = rng.random((rows, cols)) < 0.2  # few significant bits: halfway cases are frequent
    x = np.where(ties, np.round(x * 16) / 16, x)
    if cols >= 64:
        x[rng.random(rows) < 0.3, 32:64] = 0.0
    x[rng.random((rows, cols)) < 0.02] *= -0.0
    return x


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_is_exact(rows, cols, fmt, dtype):
    rng = np.random.default_rng(rows * 10007 + cols)
    x = host16(spread_values(rng, rows, cols), DTYPES[dtype])
    out = GuardedMx(rows, cols, fmt)
    got = ttc.mx_quantize(dev16(x, DTYPES[dtype], 8, 1), fmt, out.q)
    assert got is out.q
    out.check(*ref.quantize(x, fmt))


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_quantize_every_fp16_value(fmt):
    """Every finite fp16 value alone in its block, and beside the block's largest."""
    bits = np.arange(65536, dtype=np.uint16)
    v = bits.view(np.float16)
    v = v[np.isfinite(v)].astype(np.float64)
    x = np.zeros((len(v), 64))
    x[:, 5] = v
    x[:, 32:] = np.resize(v, (len(v), 32))
    x[:, 40] = v
    out = GuardedMx(*x.shape, fmt)
    ttc.mx_quantize(dev16(x, torch.float16), fmt, out.q)
    out.check(*ref.quantize(x, fmt))


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_extremes(fmt, dtype):
    t = DTYPES[dtype]
    big, small = torch.finfo(t).max, torch.finfo(t).smallest_normal
    x = np.zeros((6, 96))
    x[0, :] = big
    x[1, :] = -big
    x[1, 3] = small
    x[2, :32] = small / 4       # subnormal block: bf16's clamp to 2^-127
    x[2, 32:64] = -small
    x[3, 7] = np.inf
    x[3, 40] = np.nan
    x[4, 64] = -np.inf
    x[5, 95] = np.nan
    x = host16(x, t)
    out = GuardedMx(*x.shape, fmt)
    ttc.mx_quantize(dev16(x, t), fmt, out.q)
    out.check(*ref.quantize(x, fmt))


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_is_exact(rows, cols, fmt, dtype):
    """All codes under scales that keep the values in the output type's range, and beyond it."""
    t = DTYPES[dtype]
    rng = np.random.default_rng(rows + cols)
    codes = rng.integers(0, 256 if fmt == "mxfp8" else 16, (rows, cols)).astype(np.uint8)
    scales = rng.integers(100, 150, (rows, -(-cols // 32))).astype(np.uint8)
    scales[rng.random(scales.shape) < 0.1] = 255
    scales[rng.random(scales.shape) < 0.1] = 0
    buf = torch.full((rows + 2, (cols + 7) // 8 * 8 + 8), 7.0, dtype=t, device="cuda")
    out = buf[1:rows + 1, :cols]
    assert ttc.mx_dequantize(make_mx(codes, scales, fmt), out=out) is out
    want = ref.round_to(ref.values(codes, scales, fmt), t)
    assert np.array_equal(ref.to_np(out), want, equal_nan=True)
    out.fill_(7.0)
    assert bool((buf == 7.0).all())


# ---------------------------------------------------------------------- the norm ---

NORM_SIZES = [(1, 1), (3, 7), (2, 32), (5, 100), (1, 4096), (9, 1000), (130, 257), (4, 8192),
              (2, 16384), (3, 20001), (2, 40000)]


@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [True, False], ids=["res", "plain"])
def test_rms_norm(rows, cols, fmt, dtype, residual):
    t = DTYPES[dtype]
    rng = np.random.default_rng(rows * 31 + cols)
    x = host16(rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 6, (rows, 1))), t)
    r = host16(rng.standard_normal((rows, cols)) * 4, t) if residual else None
    w = host16(1 + 0.3 * rng.standard_normal(cols), t)
    h = ref.round_to(x + r, t) if residual else x
    want = ref.norm(h, w, 1e-5)
    kw = {}
    if fmt:
        guard = GuardedMx(rows, cols, fmt)
        kw["out"] = guard.q
    if residual:
        kw["residual"] = dev16(r, t, 16)
    got = ttc.rms_norm(dev16(x, t, 8, 1), dev_vec(w, t), 1e-5, format=fmt, **kw)
    if residual:
        got, hh = got
        assert np.array_equal(ref.to_np(hh), h)
    if fmt:
        guard.check(*ref.quantize(want, fmt))
    else:
        # the formula's value rounded once; the 64-bit reference is itself off by some 2^-50
        assert np.array_equal(ref.to_np(got), ref.round_to(want, t))


@pytest.mark.parametrize("rows,cols", [(3, 1000), (2, 40000)])
@pytest.mark.parametrize("place", ["x", "residual"])
def test_rms_norm_updates_the_stream_in_place(rows, cols, place):
    t = torch.float16
    rng = np.random.default_rng(5)
    x, r = (host16(rng.standard_normal((rows, cols)), t) for _ in range(2))
    w = host16(rng.standard_normal(cols), t)
    dx, dr = dev16(x, t), dev16(r, t)
    into = dx if place == "x" else dr
    y, h = ttc.rms_norm(dx, dev_vec(w, t), 1e-6, residual=dr, residual_out=into)
    assert h is into
    want = ref.round_to(x + r, t)
    assert np.array_equal(ref.to_np(into), want)
    assert np.array_equal(ref.to_np(dr if place == "x" else dx), r if place == "x" else x)
    assert np.array_equal(ref.to_np(y), ref.round_to(ref.norm(want, w, 1e-6), t))


@pytest.mark.parametrize("cols", [500, 40000])
def test_rms_norm_onto_its_input(cols):
    t = torch.bfloat16
    x = host16(np.random.default_rng(1).standard_normal((3, cols)), t)
    dx = dev16(x, t)
    ttc.rms_norm(dx, dev_vec(np.ones(cols), t), 0.0, out=dx)
    assert np.array_equal(ref.to_np(dx), ref.round_to(ref.norm(x, np.ones(cols), 0.0), t))


@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
def test_rms_norm_of_special_rows(fmt):
    """Zero rows, rows with an infinity or a NaN, and rows beside them."""
    t = torch.float16
    rng = np.random.default_rng(9)
    x = host16(rng.standard_normal((6, 160)), t)
    x[1] = 0.0
    x[2, 70] = np.inf
    x[3, 10] = np.nan
    x[4] = 65504.0
    w = host16(1 + 0.1 * rng.standard_normal(160), t)
    want = ref.norm(x, w, 1e-6)
    got = ttc.rms_norm(dev16(x, t), dev_vec(w, t), 1e-6, format=fmt)
    if fmt is None:
        assert np.array_equal(ref.to_np(got), ref.round_to(want, t), equal_nan=True)
    else:
        codes, scales = ref.quantize(want, fmt)
        assert np.array_equal(got.scales.cpu().numpy(), ref.tile_scales(scales, 160))
        data = got.data.cpu().numpy()[:, :ref.row_bytes(160, fmt)]
        assert np.array_equal(data, ref.pack(codes, fmt))


@pytest.mark.parametrize("rows_of_ten", [1, 30])
@pytest.mark.parametrize("cols", [100, 3000, 40000])
@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rms_norm_where_squares_leave_fp32(rows_of_ten, cols, fmt, eps):
    """bf16 rows from its smallest values to its largest, beside ordinary ones."""
    t = torch.bfloat16
    rng = np.random.default_rng(cols)
    # (with eps = 1e-6 an h this small is not scaled: kept where h w is normal in fp32)
    size = np.exp2([-131.0 if eps == 0 else -90, -80, -75, -60, -41, 0, 40, 63, 64, 125])
    size = np.tile(size, rows_of_ten)[:, None]
    x = host16(np.clip(rng.standard_normal((len(size), cols)), -3.9, 3.9) * size, t)
    r = host16(np.clip(rng.standard_normal((len(size), cols)), -3.9, 3.9) * size, t)
    w = host16(1 + 0.1 * rng.standard_normal(cols), t)
    h = ref.round_to(x + r, t)
    assert np.isfinite(h).all() and (np.abs(h).max(1) > 0).all()
    want = ref.norm(h, w, float(np.float32(eps)))
    got, hh = ttc.rms_norm(dev16(x, t), dev_vec(w, t), eps, residual=dev16(r, t), format=fmt)
    assert np.array_equal(ref.to_np(hh), h)
    if fmt is None:
        assert np.array_equal(ref.to_np(got), ref.round_to(want, t))
    else:
        codes, scales = ref.quantize(want, fmt)
        assert np.array_equal(got.scales.cpu().numpy(), ref.tile_scales(scales, cols))
        data = got.data.cpu().numpy()[:, :ref.row_bytes(cols, fmt)]
        assert np.array_equal(data, ref.pack(codes, fmt))


# --------------------------------------------------------------------- the product ---

SHAPES = [(1, 1, 1), (1, 128, 32), (2, 130, 33), (16, 128, 256), (17, 100, 100), (32, 777, 1000),
          (33, 64, 300), (64, 257, 129), (65, 128, 128), (128, 128, 512), (129, 300, 1025),
          (200, 1000, 700), (256, 256, 256), (300, 515, 2050), (513, 257, 130), (1, 1000, 8192),
          (40, 130, 16385), (65, 257, 4100), (70, 600, 4100), (129, 100, 5000),
          (200, 1000, 8200), (385, 514, 4097)]


# enough 256 x 256 tiles for the CTA-pair kernel: one wave and several, ragged
# rows and columns, K of a part of a k-block, of one and of many
LARGE = [(1300, 2100, 70), (1500, 1700, 513), (2600, 2601, 1100), (4100, 1000, 260),
         (300, 9000, 4111)]


def exact_operand(rng, rows, cols, fmt):
    """Codes and scales whose products sum exactly in 24 bits."""
    if fmt == "mxfp4":
        codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    else:  # 0, +-0.5, +-1, +-1.5, +-2, +-3
        mags = np.array([0, 0x30, 0x38, 0x3C, 0x40, 0x44], np.uint8)
        codes = mags[rng.integers(0, 6, (rows, cols))] | (rng.integers(0, 2, (rows, cols)) * 128)
        codes = codes.astype(np.uint8)
    scales = rng.integers(125, 129, (rows, -(-cols // 32))).astype(np.uint8)
    return codes, scales


@pytest.mark.parametrize("M,N,K", SHAPES + LARGE)
@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_product_of_exact_sums(M, N, K, fmt, dtype):
    """Every partial sum is a multiple of 2^-6 below 2^18, so fp32 holds it
    exactly in any order and only the output is rounded."""
    t = DTYPES[dtype]
    rng = np.random.default_rng(M + 3 * N + 7 * K)
    a, b = exact_operand(rng, M, K, fmt), exact_operand(rng, N, K, fmt)
    va, vb = ref.values(*a, fmt), ref.values(*b, fmt)
    # a 16385-long sum of products up to 144: thin out until it fits
    assert (np.abs(va) @ np.abs(vb).T).max() < 2.0 ** 18
    buf = torch.full((M + 2, (N + 7) // 8 * 8 + 8), 7.0, dtype=t, device="cuda")
    out = buf[1:M + 1, :N]
    ttc.gemm_mx(make_mx(*a, fmt), make_mx(*b, fmt), out=out)
    assert np.array_equal(ref.to_np(out), ref.round_to(va @ vb.T, t))
    out.fill_(7.0)
    assert bool((buf == 7.0).all()), "wrote outside the output"


def random_operand(rng, rows, cols, fmt, scale):
    x = rng.standard_normal((rows, cols)) * scale
    codes, scales = ref.quantize(x, fmt)
    return codes, scales


@pytest.mark.parametrize("M,N,K", [(1, 300, 700), (20, 200, 1000), (50, 129, 515), (100, 128, 2000),
                                   (300, 400, 1100), (150, 300, 4200),
                                   (1601, 1500, 640)])
@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("bias", [True, False], ids=["bias", "nobias"])
def test_product(M, N, K, fmt, dtype, act, bias):
    t = DTYPES[dtype]
    rng = np.random.default_rng(M * N + K)
    a, b = random_operand(rng, M, K, fmt, 1.0), random_operand(rng, N, K, fmt, 0.05)
    bv = host16(rng.standard_normal(N), t) if bias else None
    want, off = ref.product(ref.values(*a, fmt), ref.values(*b, fmt), bv, act)
    got = ttc.gemm_mx(make_mx(*a, fmt), make_mx(*b, fmt), None if bv is None else dev_vec(bv, t),
                      act, dtype=t)
    err = np.abs(ref.to_np(got) - want)
    assert (err <= off * (1 + ref.HALF[t]) + ref.HALF[t] * np.abs(want) + ref.TINY[t]).all()


@pytest.mark.parametrize("M", [1, 40, 200, 12000])
@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("side", ["a", "b"])
def test_nan_blocks_stay_in_their_row(M, fmt, side):
    """A NaN block makes its row (of A) or column (of B) NaN and leaves the others as they were."""
    rng = np.random.default_rng(M)
    N, K = 200, 300
    a, b = exact_operand(rng, M, K, fmt), exact_operand(rng, N, K, fmt)
    hit = a if side == "a" else b
    where = rng.choice(hit[1].shape[0], 1 + hit[1].shape[0] // 50, replace=False)
    hit[1][where, rng.integers(0, hit[1].shape[1], len(where))] = 255
    hit[0][where, :] &= 0 if M == 1 else 255  # zero elements are NaN under a NaN scale, too
    want = ref.values(*a, fmt) @ ref.values(*b, fmt).T
    assert np.isnan(want).any() and (M == 1 and side == "a" or not np.isnan(want).all())
    got = ttc.gemm_mx(make_mx(*a, fmt), make_mx(*b, fmt))
    assert np.array_equal(ref.to_np(got), ref.round_to(want, torch.float16), equal_nan=True)


@pytest.mark.parametrize("M", [3, 300, 12000])
def test_scales_from_end_to_end(M):
    """Scales far from 1 on both sides that cancel: 2^60 against 2^-60, and the smallest."""
    rng = np.random.default_rng(2)
    N, K = 140, 160
    a, b = exact_operand(rng, M, K, "mxfp8"), exact_operand(rng, N, K, "mxfp8")
    a[1][:] = a[1] + 60
    b[1][:] = b[1] - 60
    want = ref.round_to(ref.values(*a, "mxfp8") @ ref.values(*b, "mxfp8").T, torch.float16)
    got = ttc.gemm_mx(make_mx(*a, "mxfp8"), make_mx(*b, "mxfp8"))
    assert np.array_equal(ref.to_np(got), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kernel", ["fill", "split", "pair", "pair_split"])
def test_gelu_of_every_value(kernel, dtype):
    """GELU down its negative tail, in each kernel: the bias runs over all values of the type and
    the product adds 0, so what is rounded is GELU of the bias alone.

    Bound on the value before it is rounded, relative: the square in the exponent has five
    roundings of 2^-24 (the factor and its product, twice each, and the square itself), x^2 / 2
    times that, below x^2 2^-22.6; the fit 2^-20.8; exp2, the reciprocal, the coefficients and some
    ten operations 2^-24 to 2^-22 each, below 2^-19.  Beyond |x| = 40 GELU is x or 0 in fp32.
    Subnormal fp32 results are off by 2^-149, and what is flushed to 0 is below 2^-135 (half of
    bf16's smallest value is 2^-134).  The output's rounding adds half a step."""
    t = DTYPES[dtype]
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(t)
    if kernel == "pair_split":  # fewer columns: the tail, the largest values, those that are none
        v = torch.cat((v[(v < -(2.0 ** -4)) & (v > -15)], v[v > 1000][-20:], v[v < -1000][-20:],
                       v[torch.isnan(v)][::50]))
    M = {"fill": 3, "split": 2, "pair": 200, "pair_split": 70}[kernel]
    K = {"fill": 0, "split": 40, "pair": 40, "pair_split": 2100}[kernel]
    x = v.double().numpy()
    bias = dev_vec(x, t)
    if K:
        a, b = (make_mx(np.zeros((n, K), np.uint8), np.full((n, -(-K // 32)), 127, np.uint8),
                        "mxfp8") for n in (M, x.size))
    else:
        a, b = (ttc.mx_empty(n, 0, "mxfp8", "cuda") for n in (M, x.size))
    got = ttc.gemm_mx(a, b, bias, "gelu", dtype=t)
    assert torch.equal(got.view(torch.int16), got[:1].view(torch.int16).expand_as(got))
    y = ref.to_np(got[0])
    # (ref.act is right to 2^-53 of x, which is nothing in the tail; erfc is right there)
    with np.errstate(invalid="ignore"):
        want = 0.5 * x * torch.special.erfc(torch.from_numpy(-x * math.sqrt(0.5))).numpy()
    kept = np.isfinite(x)
    assert np.array_equal(y[~kept], want[~kept], equal_nan=True)  # inf, and NaN for -inf and NaN
    x, y, want = x[kept], y[kept], want[kept]
    off = np.abs(want) * (2.0 ** -18 + np.minimum(x * x, 1600) * 2.0 ** -22) + 2.0 ** -135
    assert (np.abs(y - want) <= off * (1 + ref.HALF[t]) + ref.HALF[t] * np.abs(want)
            + ref.TINY[t]).all()


def test_product_without_elements():
    for t in (torch.float16, torch.bfloat16):
        bias = dev_vec(host16(np.linspace(-2, 2, 37), t), t)
        a, b = ttc.mx_empty(5, 0, "mxfp4", "cuda"), ttc.mx_empty(37, 0, "mxfp4", "cuda")
        c = ttc.gemm_mx(a, b, bias, "relu", dtype=t)
        assert torch.equal(c, bias.clamp_min(0).expand(5, 37))
        assert not ttc.gemm_mx(a, b, dtype=t).any()


# ------------------------------------------- every kernel that a size can take ---
# (148 SMs; the norm has 4, 2 or 1 vectors a thread, or reads its rows twice; a product takes
# the split kernel, with one CTA an SM and a deep ring or two, its K in 1 to 8 parts, the pair
# split kernel in 1 to 4 parts, or the pair kernel)


@pytest.mark.parametrize("rows,cols", [(4800, 300), (2400, 1100), (620, 8000), (310, 16000)],
                         ids=["one_warp", "two_warps", "eight_warps", "sixteen_warps"])
@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rms_norm_of_many_rows(rows, cols, fmt, dtype):
    """Four vectors a thread: rows * threads a row from 1024 * 148 on."""
    test_rms_norm(rows, cols, fmt, dtype, (rows + cols) % 20 == 0)


@pytest.mark.parametrize("rows,cols", [(620, 4090), (300, 8100)])
@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("residual", [True, False], ids=["res", "plain"])
def test_rms_norm_of_some_rows(rows, cols, fmt, residual):
    """Two vectors a thread, loaded together with the weights."""
    test_rms_norm(rows, cols, fmt, "bf16", residual)


@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows,cols", [(4810, 260), (950, 4100), (480, 10000)])
def test_rms_norm_of_many_rows_where_squares_leave_fp32(rows, cols, fmt):
    """bf16 rows of every size among each other, several of them in a CTA."""
    t = torch.bfloat16
    rng = np.random.default_rng(rows)
    size = np.exp2(rng.choice([-131.0, -90, -80, -41, 0, 0, 0, 40, 63, 64, 125], rows))[:, None]
    x = host16(np.clip(rng.standard_normal((rows, cols)), -3.9, 3.9) * size, t)
    w = host16(1 + 0.1 * rng.standard_normal(cols), t)
    want = ref.norm(x, w, 0.0)
    got = ttc.rms_norm(dev16(x, t), dev_vec(w, t), 0.0, format=fmt)
    if fmt is None:
        assert np.array_equal(ref.to_np(got), ref.round_to(want, t))
    else:
        codes, scales = ref.quantize(want, fmt)
        assert np.array_equal(got.scales.cpu().numpy(), ref.tile_scales(scales, cols))
        data = got.data.cpu().numpy()[:, :ref.row_bytes(cols, fmt)]
        assert np.array_equal(data, ref.pack(codes, fmt))


# one CTA an SM, K whole, in rings of 10, 9 and 8 stages that fill and do not; then more tiles
# than SMs; then the pair split kernel in 3, 2, 1 parts and with several rows of tiles
OTHER_KERNELS = [(1, 9700, 600), (1, 9700, 4200), (4, 18900, 1300), (16, 14336, 3000),
                 (20, 12000, 300), (32, 9601, 3000), (40, 10000, 300), (64, 12345, 2100),
                 (128, 9473, 1000), (20, 20000, 300), (3, 28672, 700), (100, 20000, 500),
                 (70, 5000, 4200), (70, 8000, 4200), (100, 12000, 4200), (200, 4000, 4200),
                 (129, 6000, 4300), (256, 4096, 4200)]


@pytest.mark.parametrize("M,N,K", OTHER_KERNELS)
@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_product_of_exact_sums_in_every_kernel(M, N, K, fmt):
    test_product_of_exact_sums(M, N, K, fmt, "bf16" if (M + N) % 2 else "fp16")


@pytest.mark.parametrize("parts", range(1, 9))
@pytest.mark.parametrize("M", [2, 15, 30, 59])
@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_product_in_any_number_of_parts(parts, M, fmt):
    """K in 1 to 8 parts of four k-blocks and a few more, read (2 rows) and sent, rows that the
    parts do not divide evenly."""
    K = (4 * parts + min(parts, 3)) * (128 if fmt == "mxfp8" else 256) - 40
    test_product_of_exact_sums(M, 200, K, fmt, "fp16")


@pytest.mark.parametrize("M,N,K", [(5, 10000, 1500), (33, 9999, 1500), (70, 5000, 4200),
                                   (90, 8000, 2100), (100, 10001, 4200)])
@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("act", ["relu", "gelu"])
def test_product_with_bias_in_every_kernel(M, N, K, fmt, act):
    test_product(M, N, K, fmt, "bf16" if K == 1500 else "fp16", act, True)


# -------------------------------------------------------------- together, in use ---


@pytest.mark.parametrize("M", [1, 24, 300])
@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_mlp_of_mx_operators(M, fmt):
    """norm(x + r) -> up projection with bias and GELU -> quantise -> down projection, whose
    output is the next residual: every step against the reference on that step's own inputs."""
    t = torch.float16
    rng = np.random.default_rng(M)
    D, F = 320, 1000
    x, r = (host16(rng.standard_normal((M, D)), t) for _ in range(2))
    g = host16(1 + 0.1 * rng.standard_normal(D), t)
    up, down = host16(0.05 * rng.standard_normal((F, D)), t), host16(0.05 * rng.standard_normal((D, F)), t)
    bias = host16(0.1 * rng.standard_normal(F), t)
    q_up, q_down = (ttc.mx_quantize(dev16(w, t), fmt) for w in (up, down))
    y, h = ttc.rms_norm(dev16(x, t), dev_vec(g, t), 1e-6, residual=dev16(r, t), format=fmt)
    u = ttc.gemm_mx(y, q_up, dev_vec(bias, t), "gelu")
    v = ttc.mx_quantize(u, fmt)
    z = ttc.gemm_mx(v, q_down)
    y2, h2 = ttc.rms_norm(z, dev_vec(g, t), 1e-6, residual=h, format=fmt)

    def close(got, want, off):
        err = np.abs(ref.to_np(got) - want)
        return (err <= off * (1 + ref.HALF[t]) + ref.HALF[t] * np.abs(want) + ref.TINY[t]).all()

    wh = ref.round_to(x + r, t)
    wy = ref.values(*ref.quantize(ref.norm(wh, g, 1e-6), fmt), fmt)
    assert np.array_equal(ref.to_np(ttc.mx_dequantize(y)), wy)
    wup, wdown = (ref.values(*ref.quantize(w, fmt), fmt) for w in (up, down))
    assert close(u, *ref.product(wy, wup, bias, "gelu"))
    wv = ref.values(*ref.quantize(ref.to_np(u), fmt), fmt)
    assert close(z, *ref.product(wv, wdown, None, "none"))
    wh2 = ref.round_to(ref.to_np(z) + wh, t)
    assert np.array_equal(ref.to_np(h2), wh2)
    wy2 = ref.values(*ref.quantize(ref.norm(wh2, g, 1e-6), fmt), fmt)
    assert np.array_equal(ref.to_np(ttc.mx_dequantize(y2)), wy2)


def test_streams_and_graph_replay():
    """Calls on two streams at once, and a captured chain replayed on new inputs, give the bits of
    plain calls."""
    t = torch.float16
    rng = np.random.default_rng(4)
    M, N, K = 24, 500, 640
    xs = [dev16(host16(rng.standard_normal((M, K)), t), t) for _ in range(4)]
    w = ttc.mx_quantize(dev16(host16(0.05 * rng.standard_normal((N, K)), t), t), "mxfp4")
    g = dev_vec(np.ones(K), t)

    def chain(x, stream=None):
        return ttc.gemm_mx(ttc.rms_norm(x, g, format="mxfp4", stream=stream), w, act="relu",
                           stream=stream)

    want = [chain(x).clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(12):
        got.append((i % 4, chain(xs[i % 4], streams[i % 2])))
    torch.cuda.synchronize()
    for i, c in got:
        assert torch.equal(c, want[i])
    static = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = chain(static)
    for x, v in zip(xs, want):
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, v)


def test_threads_on_their_own_streams():
    """Four host threads, each on a stream of its own, calling every operator at once."""
    import threading
    t = torch.float16
    rng = np.random.default_rng(21)
    g = dev_vec(host16(1 + 0.1 * rng.standard_normal(384), t), t)
    weights = [ttc.mx_quantize(dev16(host16(0.05 * rng.standard_normal((n, 384)), t), t), "mxfp8")
               for n in (200, 3000)]
    xs = [dev16(host16(rng.standard_normal((m, 384)), t), t) for m in (1, 30, 100, 1000)]

    def chain(x):
        q = ttc.rms_norm(x, g, format="mxfp8")
        return [ttc.mx_dequantize(q)] + [ttc.gemm_mx(q, w, act="gelu") for w in weights]

    want = [chain(x) for x in xs]
    torch.cuda.synchronize()
    errors = []

    def worker(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got = [(i, chain(xs[i])) for _ in range(5) for i in ((k + j) % 4 for j in range(4))]
                stream.synchronize()
            for i, c in got:
                if not all(torch.equal(u, v) for u, v in zip(c, want[i])):
                    errors.append((k, i))
        except Exception as e:
            errors.append((k, repr(e)))

    threads = [threading.Thread(target=worker, args=(k,)) for k in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=120)
    assert not any(th.is_alive() for th in threads) and not errors, errors


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_offsets_past_32_bits(fmt):
    """Inputs and outputs of more than 2^32 bytes: the first and last rows and some between."""
    t = torch.bfloat16
    rows, cols = 66000, 33000
    x = torch.zeros((rows, cols), dtype=t, device="cuda")
    pick = [0, 1, 65, 32768, 65075, 65076, rows - 130, rows - 1]  # 65076 x 33000 passes 2^31
    rng = np.random.default_rng(0)
    v = host16(rng.standard_normal((len(pick), cols)), t)
    x[pick] = torch.from_numpy(v).to(t).cuda()
    q = ttc.mx_quantize(x, fmt)
    codes, scales = ref.quantize(v, fmt)
    assert np.array_equal(q.data[pick].cpu().numpy()[:, :ref.row_bytes(cols, fmt)],
                          ref.pack(codes, fmt))
    blocks = ttc.mx_untile_scales(q.scales, rows, cols)[pick].cpu().numpy()
    assert np.array_equal(blocks, scales)
    x.fill_(1.0)
    ttc.mx_dequantize(q, out=x)
    assert np.array_equal(ref.to_np(x[pick]), ref.values(codes, scales, fmt))
    w = dev_vec(np.ones(cols), t)
    y = ttc.rms_norm(x, w, 1e-6, out=x)
    assert np.array_equal(ref.to_np(y[pick]),
                          ref.round_to(ref.norm(ref.values(codes, scales, fmt), np.ones(cols), 1e-6), t))
    del x, y, q
    # C of 66000 x 33000
    K = 64
    a = np.zeros((rows, K), np.uint8)
    sa = np.full((rows, 2), 127, np.uint8)
    small, one = exact_operand(rng, len(pick), K, fmt), exact_operand(rng, cols, K, fmt)
    a[pick], sa[pick] = small
    c = ttc.gemm_mx(make_mx(a, sa, fmt), make_mx(*one, fmt), dtype=t)
    want = ref.values(*small, fmt) @ ref.values(*one, fmt).T
    assert np.array_equal(ref.to_np(c[pick]), ref.round_to(want, t))
    assert int((c != 0).any(1).sum()) <= len(pick)


@pytest.mark.parametrize("cols", [300, 20000])
def test_rms_norm_without_keeping_the_sum(cols):
    """The C entry point with a residual and no place for h."""
    t = torch.float16
    rng = np.random.default_rng(cols)
    x, r = (host16(rng.standard_normal((5, cols)), t) for _ in range(2))
    w = host16(1 + 0.1 * rng.standard_normal(cols), t)
    dx, dr, dw, y = dev16(x, t), dev16(r, t), dev_vec(w, t), dev16(np.zeros((5, cols)), t)
    ld = dx.stride(0)
    assert raw("mx_rms_norm", dx.data_ptr(), dr.data_ptr(), dw.data_ptr(), None, y.data_ptr(), None,
               5, cols, ld, ld, 0, ld, 1e-6, 0, 0) == 0
    h = ref.round_to(x + r, t)
    eps = float(np.float32(1e-6))
    assert np.array_equal(ref.to_np(y), ref.round_to(ref.norm(h, w, eps), t))
    assert np.array_equal(ref.to_np(dx), x) and np.array_equal(ref.to_np(dr), r)


def test_same_bits_on_every_run():
    rng = np.random.default_rng(11)
    a = make_mx(*random_operand(rng, 40, 5000, "mxfp8", 1.0), "mxfp8")
    b = make_mx(*random_operand(rng, 700, 5000, "mxfp8", 1.0), "mxfp8")
    c = ttc.gemm_mx(a, b)
    for _ in range(20):
        assert torch.equal(ttc.gemm_mx(a, b), c)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("M", [1, 2, 3, 4])
def test_few_rows_back_to_back(M, fmt):
    """Up to 4 rows with K divided read the parts from the other CTAs' shared memory: launch
    after launch, products of two shapes in turn, each with the sums of its own operands (exact
    in fp32, so equal bits)."""
    rng = np.random.default_rng(100 + M)
    cases = []
    for N, K in ((300, 2000), (1000, 4100), (130, 8200)):
        a, b = exact_operand(rng, M, K, fmt), exact_operand(rng, N, K, fmt)
        want = ref.round_to(ref.values(*a, fmt) @ ref.values(*b, fmt).T, torch.float16)
        out = torch.empty((40, M, (N + 7) // 8 * 8), dtype=torch.float16, device="cuda")
        cases.append((make_mx(*a, fmt), make_mx(*b, fmt), want, out, N))
    for i in range(40):
        for a, b, _, out, N in cases:
            ttc.gemm_mx(a, b, out=out[i, :, :N])
    for _, _, want, out, N in cases:
        for i in range(40):
            assert np.array_equal(ref.to_np(out[i, :, :N]), want), (N, i)


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_pair_tiles_back_to_back(fmt):
    """The CTA-pair kernel launch after launch, shapes in turn with 1 to 5 tiles a pair (each
    buffer of the accumulator last, and not handed back), the last rows and columns nearly empty
    (warps with nothing to store)."""
    rng = np.random.default_rng(77)
    K = 96
    cases = []
    for M, N in ((257, 9300), (1537, 2700), (2305, 4400), (3841, 4900), (4609, 4700)):
        a, b = exact_operand(rng, M, K, fmt), exact_operand(rng, N, K, fmt)
        want = torch.as_tensor(ref.round_to(ref.values(*a, fmt) @ ref.values(*b, fmt).T,
                                            torch.float16)).half().cuda()
        out = torch.empty((M, (N + 7) // 8 * 8), dtype=torch.float16, device="cuda")[:, :N]
        cases.append((make_mx(*a, fmt), make_mx(*b, fmt), want, out,
                      torch.ones((), dtype=torch.bool, device="cuda")))
    for _ in range(10):
        for a, b, want, out, same in cases:
            ttc.gemm_mx(a, b, out=out)
        for a, b, want, out, same in cases:
            same &= (out == want).all()
            out.fill_(7.0)
    assert all(bool(c[4]) for c in cases)


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_pairs_whose_ring_does_not_fill(fmt):
    """Both CTA-pair kernels with fewer k-blocks than ring stages, as many and some more, launch
    after launch: producers leave only after every stage they filled has been released."""
    rng = np.random.default_rng(78)
    step = 128 if fmt == "mxfp8" else 256  # elements of a k-block
    cases = []
    for M, N, blocks in [(300, 9500, n) for n in (1, 5, 6, 7, 12, 13)] + \
                        [(70, 300, n) for n in (16, 31, 32, 33, 35)]:
        K = blocks * step - 7
        a, b = exact_operand(rng, M, K, fmt), exact_operand(rng, N, K, fmt)
        want = ref.round_to(ref.values(*a, fmt) @ ref.values(*b, fmt).T, torch.float16)
        cases.append((make_mx(*a, fmt), make_mx(*b, fmt), torch.as_tensor(want).half().cuda()))
    got = []
    for _ in range(5):
        got.append([ttc.gemm_mx(a, b) for a, b, _ in cases])
    for outs in got:
        for c, (_, _, want) in zip(outs, cases):
            assert torch.equal(c, want)


# -------------------------------------------------------------------------- refusals ---


def raw(name, *args):
    return getattr(ttc.mx_lib(), name)(*args, torch.cuda.current_stream().cuda_stream)


def test_refusals_of_pointers_and_strides():
    """Misaligned, host, foreign or too short buffers are refused before a launch."""
    x = torch.zeros(8, 64, dtype=torch.float16, device="cuda")
    d = torch.zeros(8, 64, dtype=torch.uint8, device="cuda")
    s = torch.zeros(512, dtype=torch.uint8, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    c = torch.zeros(8, 8, dtype=torch.float16, device="cuda")
    X, D, S, W, C = (t.data_ptr() for t in (x, d, s, w, c))
    host = torch.zeros(4096, dtype=torch.uint8)
    H = (host.data_ptr() + 15) // 16 * 16

    def quantize(x=X, q=D, sc=S, rows=8, cols=64, ldx=64, ldq=64):
        return raw("mx_quantize", x, q, sc, rows, cols, ldx, ldq, 0, 1)

    assert quantize() == 0
    assert quantize(x=X + 2) == -2 and quantize(q=D + 4) == -2 and quantize(sc=S + 1) == -2
    assert quantize(ldx=68, cols=60) == -2 and quantize(ldq=72) == -2
    assert quantize(ldx=56) == -1 and quantize(ldq=48) == -1
    for bad in (0, H):
        assert quantize(x=bad) == -1 and quantize(q=bad) == -1 and quantize(sc=bad) == -1
    assert quantize(rows=1 << 24, ldx=1 << 20) == -1  # far past the allocation
    assert raw("mx_dequantize", D, S, H, 8, 64, 64, 64, 0, 1) == -1

    def norm(x=X, r=None, wt=W, h=None, y=C, sc=S, rows=1, cols=64, fmt=0, ldy=64):
        return raw("mx_rms_norm", x, r, wt, h, y, sc, rows, cols, 64, 64, 64, ldy, 1e-6, 0, fmt)

    y2 = torch.zeros(8, 64, dtype=torch.float16, device="cuda")
    Y = y2.data_ptr()
    assert norm(y=Y, rows=8) == 0
    assert norm(y=Y, wt=W + 2) == -2 and norm(y=Y, wt=0) == -1 and norm(y=Y, wt=H) == -1
    assert norm(y=X) == 0                                # onto its input: allowed
    assert norm(y=X, r=Y) == -1                          # but not with a residual
    assert norm(y=Y, r=Y) == -1 and norm(y=Y, r=X, h=Y) == -1
    assert norm(y=X, fmt=1) == -1                        # nor to MX
    assert norm(y=D, fmt=1, sc=0) == -1 and norm(y=D, fmt=2, sc=S + 8) == -2

    def gemm(a=D, sa=S, b=D, sb=S, bias=None, out=C, K=64, lda=64, ldc=8):
        return raw("mx_gemm", a, sa, b, sb, bias, out, 8, 8, K, lda, 64, ldc, 1, 0, 0)

    assert gemm() == 0
    assert gemm(a=D + 8) == -2 and gemm(sb=S + 8) == -2 and gemm(out=C + 2) == -2
    assert gemm(bias=W + 2) == -2 and gemm(bias=H) == -1
    assert gemm(lda=56) == -1 and gemm(lda=72) == -2 and gemm(ldc=12) == -2
    for bad in (0, H):
        assert gemm(a=bad) == -1 and gemm(sa=bad) == -1 and gemm(out=bad) == -1
    torch.cuda.synchronize()


def test_refusals_of_extents_past_64_bits():
    """Rows and strides whose product passes 2^64 and comes back as a few bytes; everything else
    about the calls is in order (scales and single rows lie in a buffer that holds them)."""
    n, ld16, ld8 = (1 << 25) + 1, 1 << 38, 1 << 39  # n rows of 2^39 bytes: 2^64 and a row
    buf = torch.zeros(1 << 29, dtype=torch.uint8, device="cuda")
    S, row, P = (buf.data_ptr() + (k << 27) for k in (0, 2, 3))
    assert ttc.mx_scale_bytes(n, 32) <= 2 << 27 and 2 * n <= 1 << 27
    Q, W, R, small = (P + k * 65536 for k in (1, 2, 3, 4))
    for fmt in (1, 2):
        assert raw("mx_quantize", P, Q, S, n, 32, ld16, ld8, 0, fmt) == -1
        assert raw("mx_dequantize", Q, S, P, n, 32, ld8, ld16, 0, fmt) == -1
        assert raw("mx_rms_norm", P, None, W, None, Q, S, n, 32, ld16, 0, 0, ld8, 1e-6, 0, fmt) == -1
        assert raw("mx_gemm", P, S, Q, small, None, R, n, 8, 32, ld8, 32, ld16, fmt, 0, 0) == -1
        assert raw("mx_gemm", P, small, Q, S, None, row, 1, n, 32, 32, ld8, n + 7, fmt, 0, 0) == -1
        assert raw("mx_gemm", P, S, Q, small, None, R, n, 8, 0, ld8, 32, ld16, fmt, 0, 0) == -1
    assert raw("mx_rms_norm", P, None, W, None, Q, None, n, 32, ld16, 0, 0, ld16, 1e-6, 0, 0) == -1
    assert raw("mx_rms_norm", P, R, W, R, Q, None, n, 32, ld16, ld16, ld16, ld16, 1e-6, 0, 0) == -1
    torch.cuda.synchronize()
    assert not buf.any()


def test_refusals_of_fp16_extents_past_64_bits():
    """The same of the fp16 products and the activation, which share the checks."""
    from tiled_tensor_core_05_b200 import ops
    lib, n, ld = ops.lib(), (1 << 25) + 1, 1 << 38
    buf = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    row, P = buf.data_ptr(), buf.data_ptr() + (1 << 27)
    Q, C = P + 65536, P + 131072
    stream = torch.cuda.current_stream().cuda_stream

    def general(A, B, out, M, N, K, lda, ldb, ldc, ta=0, tb=0):
        return lib.gemm_f16_general(A, B, None, out, M, N, K, lda, ldb, ldc, ta, tb, 0, 0, stream)

    assert general(P, Q, C, n, 32, 32, ld, 32, ld) == -1
    assert general(P, Q, C, n, 32, 0, 32, 32, ld) == -1       # nothing but the output
    assert general(row, Q, C, 1, 32, n, n + 7, ld, 32) == -1
    assert general(P, Q, C, 32, 32, n, ld, ld, 32, ta=1) == -1
    assert general(P, Q, row, 1, n, 32, 32, ld, n + 7, tb=1) == -1
    assert lib.gemm_activation_f32(P, C, 1 << 62, 1, stream) == -1
    assert lib.gemm_activation_f32(P, C, (1 << 62) + 8, 2, stream) == -1
    torch.cuda.synchronize()
    assert not buf.any()


@pytest.mark.parametrize("library", ["mx", "fp16"])
def test_failed_status_query_is_not_reported_again(library):
    """The status of a stream that is being captured cannot be read; the error is that call's, not
    the next one's, whose kernel runs."""
    import ctypes
    from tiled_tensor_core_05_b200 import ops
    rt = ctypes.CDLL("libcudart.so.12")  # torch's, as it is loaded
    stream = torch.cuda.Stream()
    handle = ctypes.c_void_p(stream.cuda_stream)
    x = torch.randn(8, 64, device="cuda").half()
    want = ttc.mx_quantize(x, "mxfp8") if library == "mx" else ops.gemm_f16(x, x.t().contiguous())
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(handle, 2) == 0  # relaxed mode
    with pytest.raises(RuntimeError):
        (ttc.mx_device_status if library == "mx" else ops.device_status)(stream=stream)
    graph = ctypes.c_void_p()
    rt.cudaStreamEndCapture(handle, ctypes.byref(graph))  # (the query has ended the capture)
    assert not graph.value
    rt.cudaGetLastError()
    if library == "mx":
        got = ttc.mx_quantize(x, "mxfp8")
        assert torch.equal(got.data, want.data) and torch.equal(got.scales, want.scales)
        assert ttc.mx_device_status() == 0
    else:
        assert torch.equal(ops.gemm_f16(x, x.t().contiguous()), want)
        assert ops.device_status() == 0


def test_refusals_of_the_python_layer():
    t = torch.float16
    x = torch.zeros(8, 64, dtype=t, device="cuda")
    w = torch.ones(64, dtype=t, device="cuda")
    q8, q4 = ttc.mx_quantize(x, "mxfp8"), ttc.mx_quantize(x, "mxfp4")
    with pytest.raises(ValueError):
        ttc.gemm_mx(q8, q4)                              # two formats
    with pytest.raises(ValueError):
        ttc.gemm_mx(q8, ttc.mx_quantize(x[:, :32], "mxfp8"))  # two inner sizes
    with pytest.raises(TypeError):
        ttc.gemm_mx(q8, q8, w[:8].bfloat16())
    with pytest.raises(ValueError):
        ttc.gemm_mx(q8, q8, w[:7])
    with pytest.raises(TypeError):
        ttc.gemm_mx(q8, q8, dtype=torch.float32)
    with pytest.raises(KeyError):
        ttc.gemm_mx(q8, q8, act="tanh")
    with pytest.raises(ValueError):
        ttc.mx_quantize(x, "mxfp8", q4)
    with pytest.raises(ValueError):
        ttc.rms_norm(x, w[:32])
    with pytest.raises(TypeError):
        ttc.rms_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        ttc.rms_norm(x, w, residual_out=x)
    with pytest.raises(ValueError):
        ttc.rms_norm(x, w, residual=x[:4])
    with pytest.raises(ValueError):
        ttc.mx_quantize(x.t(), "mxfp8")                  # columns apart
    with pytest.raises(RuntimeError):
        ttc.mx_quantize(x[:1].expand(8, 64), "mxfp8")    # rows on top of each other
    with pytest.raises(RuntimeError):
        ttc.mx_quantize(x[:, 1:], "mxfp8")               # rows not on 16 bytes
