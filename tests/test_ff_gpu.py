"""The feed-forward operators on the GPU against the plain 64-bit implementation of
``ff_ref``: bit by bit where all sums are exact, within derived bounds otherwise."""
import threading
import zlib

import pytest
import torch

import ff_ref as ref
import tiled_tensor_core_05_b200 as ttc

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    ttc.ff_lib()
    yield
    torch.cuda.synchronize()
    assert ttc.ff_device_status() == 0


def gen(*key):
    g = torch.Generator()
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def dev(x, dtype, pad_cols=0, pad_rows=0):
    """A device matrix of x's values with NaN around it."""
    rows, cols = x.shape
    unit = 16 // torch.tensor([], dtype=dtype).element_size()
    buf = torch.full((rows + pad_rows, -(-cols // unit) * unit + pad_cols), float("nan"),
                     dtype=dtype, device="cuda")
    buf[:rows, :cols] = x.to(dtype).cuda()
    return buf[:rows, :cols]


class Out:
    """A device output whose surroundings hold a canary."""

    def __init__(self, rows, cols, dtype):
        self.buf = torch.full((rows + 2, (cols + 7) // 8 * 8 + 8), -77.0, dtype=dtype,
                              device="cuda")
        self.view = self.buf[1:rows + 1, :cols]

    def check(self, what=""):
        left = self.buf.clone()
        left[1:self.view.shape[0] + 1, :self.view.shape[1]] = -77.0
        assert (left == -77.0).all(), f"{what}: wrote outside"


def integers(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g).double()


def normal(g, dtype, *shape, std=1.0):
    """N(0, std^2) rounded to the type, as fp64."""
    return (torch.randn(shape, generator=g) * std).to(dtype).double()


GATED = [(1, 1, 1), (1, 8, 64), (2, 100, 70), (4, 64, 64), (5, 65, 63), (16, 64, 200),
         (17, 130, 200), (33, 200, 1000), (64, 512, 4096), (65, 300, 500), (130, 129, 257),
         (200, 1000, 1000), (257, 700, 136), (300, 5000, 520), (1400, 1800, 72), (2000, 4001, 33)]


# ------------------------------------------------------------------- gated, forward ---


@pytest.mark.parametrize("M,F,D", GATED)
@pytest.mark.parametrize("name", ["none", "relu"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_exact(M, F, D, name, dtype):
    """Small integers: sums are exact, h is rounded once, and gate and up are the sums."""
    t = DTYPES[dtype]
    g = gen(M, F, D, name)
    x, wg, wu = (integers(g, -2, 2, *s) for s in ((M, D), (F, D), (F, D)))
    r = ref.Gated(x, wg, wu, name)
    out = Out(M, F, t)
    args = dev(x, t, 8, 1), dev(wg, t, 0, 1), dev(wu, t, 16, 1)
    got, gate, up = ttc.gemm_gated(*args, name, out.view, save=True)
    assert got is out.view
    assert torch.equal(got.cpu(), ref.rounded(r.h, t))
    assert torch.equal(gate.cpu().double(), r.g) and torch.equal(up.cpu().double(), r.u)
    out.check()
    assert torch.equal(ttc.gemm_gated(*args, name), got)  # the same bits, without the sums


@pytest.mark.parametrize("M,F,D", [s for s in GATED if s[0] * s[1] * s[2] < 3e8])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_random(M, F, D, name, dtype):
    t = DTYPES[dtype]
    g = gen(M, F, D, name, dtype)
    x = normal(g, t, M, D, std=2.0)
    wg, wu = (normal(g, t, F, D, std=2.0 / D ** 0.5) for _ in range(2))
    r = ref.Gated(x, wg, wu, name)
    h = ttc.gemm_gated(dev(x, t), dev(wg, t), dev(wu, t), name)
    ref.close(h, r.h, r.h_bound(t), f"{M} x {F} x {D} {name}")


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_gated_every_value(M, name, dtype):
    """Each finite value of the type as the gate's sum, in a product with 1: the activation in each
    kernel's epilogue, down its tails."""
    t = DTYPES[dtype]
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(t)
    v = v[v.float().abs() < 1e30]
    # one row takes every seventh value or so; 300 take some more than once, in enough tiles for the
    # kernel of large products
    F = {1: 8192, 300: 2560}.get(M, -(-v.numel() // M))
    step = max(1, v.numel() // (M * F))
    gate = v[::step].repeat(-(-M * F * step // v.numel()) + 1)[:M * F].view(M, F)
    # row m of x picks column m of the weights: gate sums are the values themselves
    x = torch.eye(M, dtype=torch.float64)
    h = ttc.gemm_gated(dev(x, t), dev(gate.t().contiguous().double(), t),
                       dev(torch.ones(F, M, dtype=torch.float64), t), name)
    want = ref.act(gate.double(), name)
    bound = ref.act_error(gate.double(), name) * want.abs() * (1 + ref.HALF[t]) + \
        ref.HALF[t] * want.abs() + ref.TINY[t]
    if name == "silu":  # the sigmoid is 0 where 2^126 is exceeded
        bound = bound + (gate.double() < -87.0) * 2e-36
    if name == "gelu":  # what the exponential flushes
        bound = bound + (gate.double() < -12.0) * 2e-36
    ref.close(h, want, bound, name)


@pytest.mark.parametrize("M", [1, 20, 600])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_special_values(M, dtype):
    """NaN and infinities reach the row or the column that they are in, and nothing else."""
    t = DTYPES[dtype]
    g = gen("special", M)
    F, D = 900, 200
    x, wg, wu = (normal(g, t, *s) for s in ((M, D), (F, D), (F, D)))
    base = ttc.gemm_gated(dev(x, t), dev(wg, t), dev(wu, t)).cpu()
    wg2, wu2 = wg.clone(), wu.clone()
    wg2[7, 3], wu2[11, 199], wg2[899, 0] = float("nan"), float("inf"), float("-inf")
    got = ttc.gemm_gated(dev(x, t), dev(wg2, t), dev(wu2, t)).cpu()
    keep = torch.ones(F, dtype=torch.bool)
    keep[[7, 11, 899]] = False
    assert torch.equal(got[:, keep], base[:, keep])
    assert got[:, 7].isnan().all()
    assert (~got[:, 11].isfinite() | (x[:, 199] == 0)).all()
    x2 = x.clone()
    x2[M - 1, 5] = float("nan")
    got = ttc.gemm_gated(dev(x2, t), dev(wg, t), dev(wu, t)).cpu()
    assert got[M - 1].isnan().all() and torch.equal(got[:M - 1], base[:M - 1])


# ------------------------------------------------------------------ gated, backward ---


@pytest.mark.parametrize("M,F,D", GATED)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["none", "relu"])
def test_gated_backward_exact(M, F, D, dtype, name):
    """Small integers: the gradients of the projections are exact in 16 bits and so are the sums."""
    t = DTYPES[dtype]
    g = gen("backward", M, F, D, name)
    # one nonzero in eight, so that |gate|, |up| times |dh| stay below 256
    x, wg, wu = (integers(g, -1, 1, *s) * (torch.rand(s, generator=g) < 0.125)
                 for s in ((M, D), (F, D), (F, D)))
    dh = integers(g, -2, 2, M, F)
    r = ref.Gated(x, wg, wu, name)
    want = r.backward(dh, t)
    assert max(r.dg.abs().max(), r.du.abs().max()) <= 256
    args = dev(x, t, 8), dev(wg, t, 0, 1), dev(wu, t, 16)
    _, gate, up = ttc.gemm_gated(*args, name, save=True)
    got = ttc.gemm_gated_backward(dev(dh, t, 8), *args, gate, up, name)
    for v, (k, (w, _)) in zip(got, want.items()):
        assert torch.equal(v.cpu(), ref.rounded(w, t)), k


@pytest.mark.parametrize("M,F,D", [(1, 8, 64), (5, 65, 63), (40, 200, 300), (257, 700, 136),
                                   (300, 1000, 520)])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_backward_random(M, F, D, name, dtype):
    t = DTYPES[dtype]
    g = gen("gradients", M, F, D, name, dtype)
    x = normal(g, t, M, D, std=2.0)
    wg, wu = (normal(g, t, F, D, std=2.0 / D ** 0.5) for _ in range(2))
    dh = normal(g, t, M, F, std=0.3)
    r = ref.Gated(x, wg, wu, name)
    args = dev(x, t), dev(wg, t), dev(wu, t)
    _, gate, up = ttc.gemm_gated(*args, name, save=True)
    got = ttc.gemm_gated_backward(dev(dh, t), *args, gate, up, name)
    for v, (k, (w, bound)) in zip(got, r.backward(dh, t).items()):
        ref.close(v, w, bound, f"{k} {M} x {F} x {D} {name}")
        # The roundings of dg and du are as large as the result's own and independent of it: the
        # result is sqrt(2) times as far off as one rounding; an error of one rounding of a
        # gradient's factor would make it sqrt(3).  10 % more for the sample: the M F squared errors
        # of dg are dg^2 (a product of three near-normal factors, E dg^4 = 27 (E dg^2)^2) times the
        # square of a uniform number (E = 1.8 E^2): their sum has a relative deviation of
        # sqrt((27 * 1.8 - 1) / (M F)), 7.7 % from 8000 values on, so the norm of both errors one of
        # 7.7 % / 4, and 10 % are five of them.  Below that number nothing follows.
        if M * F >= 8000:
            once = (ref.rounded(w, t).double() - w).norm()
            assert (v.cpu().double() - w).norm() <= 1.1 * 2 ** 0.5 * once + 2.0 ** -17 * w.norm(), k


def test_gated_backward_against_differences():
    """d loss / d x along a direction, by central differences of the fp64 definition."""
    t = torch.bfloat16
    g = gen("differences")
    M, F, D = 30, 200, 96
    x, wg, wu = normal(g, t, M, D), normal(g, t, F, D, std=0.15), normal(g, t, F, D, std=0.15)
    dh = normal(g, t, M, F)
    for name in ("silu", "gelu", "none"):
        args = dev(x, t), dev(wg, t), dev(wu, t)
        _, gate, up = ttc.gemm_gated(*args, name, save=True)
        got = ttc.gemm_gated_backward(dev(dh, t), *args, gate, up, name)
        for i, v in enumerate((x, wg, wu)):
            d = torch.randn(v.shape, generator=g, dtype=torch.float64)
            eps, loss = 1e-4, []
            for sign in (1, -1):
                p = [x, wg, wu]
                p[i] = v + sign * eps * d
                loss.append((ref.Gated(*p, name).h * dh).sum())
            want = (loss[0] - loss[1]) / (2 * eps)
            along = (got[i].cpu().double() * d).sum()
            # independent errors of half a step (2^-8) of each gradient: below 2^-7 of the norm of
            # the terms, at 4 deviations; the differences' own error is of order eps^2
            assert abs(along - want) <= 2.0 ** -7 * (got[i].cpu().double() * d).norm() * 4 + 1e-5


def test_gated_backward_parts():
    """Only what is needed is computed, with the same bits."""
    t = torch.float16
    g = gen("parts")
    x, wg, wu, dh = (normal(g, t, *s) for s in ((50, 72), (300, 72), (300, 72), (50, 300)))
    args = dev(x, t), dev(wg, t), dev(wu, t)
    _, gate, up = ttc.gemm_gated(*args, save=True)
    full = ttc.gemm_gated_backward(dev(dh, t), *args, gate, up)
    only_x = ttc.gemm_gated_backward(dev(dh, t), *args, gate, up, need_w=False)
    only_w = ttc.gemm_gated_backward(dev(dh, t), *args, gate, up, need_x=False)
    assert torch.equal(only_x[0], full[0]) and only_x[1:] == (None, None)
    assert only_w[0] is None and all(torch.equal(a, b) for a, b in zip(only_w[1:], full[1:]))
    none = ttc.gemm_gated_backward(dev(dh, t), *args, gate, up, need_x=False, need_w=False)
    assert none == (None, None, None)


# ------------------------------------------------------------------- 4-bit weights ---


class W4:
    """Random codes, scales and zero points on the host and, with canaries, on the device."""

    def __init__(self, g, rows, cols, group, zeros, dtype, exact=False):
        groups = -(-cols // group)
        self.codes = torch.randint(0, 16, (rows, cols), generator=g)
        if exact:  # powers of two
            s = torch.exp2(torch.randint(-2, 2, (groups, rows), generator=g).double())
        else:
            s = torch.randn((groups, rows), generator=g).double() * 0.1
        self.scales = s.to(dtype).double()
        self.zeros = torch.randint(0, 16, (groups, rows), generator=g) if zeros else None
        self.value = ref.weight(self.codes, self.scales, self.zeros, group)
        words = ref.pack_words(self.codes, fill=9)
        data = torch.full((rows + 1, -(-words.shape[1] // 16) * 16 + 16), 0xA5, dtype=torch.uint8)
        data[:rows, :words.shape[1]] = words
        z = None
        if zeros:
            z = torch.full((groups + 1, -(-rows // 16) * 16 + 16), 0xFF, dtype=torch.uint8)
            z[:groups, :rows] = self.zeros.to(torch.uint8)
            z = z.cuda()[:groups, :rows]
        self.w = ttc.W4Tensor(data.cuda()[:rows, :words.shape[1]], dev(self.scales, dtype, 8, 1), z,
                              rows, cols, group)


W4_SIZES = [(1, 1, 1), (1, 64, 7), (2, 100, 31), (3, 128, 33), (4, 129, 256), (5, 1000, 1000),
            (8, 300, 257), (9, 200, 520), (16, 128, 4096), (17, 70, 100), (32, 513, 1030),
            (33, 130, 64), (64, 256, 2048), (65, 100, 300), (150, 64, 96), (1, 5000, 4100)]


@pytest.mark.parametrize("M,N,K", W4_SIZES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_w4_exact(M, N, K, group, zeros, dtype):
    """Integers, and scales that are powers of two: every sum is exact."""
    t = DTYPES[dtype]
    g = gen("w4", M, N, K, group, zeros)
    x = integers(g, -3, 3, M, K)
    w = W4(g, N, K, group, zeros, t, exact=True)
    bias = integers(g, -8, 8, N)
    out = Out(M, N, t)
    xd = dev(x, t, 8, 1)
    got = ttc.gemm_w4(xd, w.w, out=out.view)
    want = x @ w.value.t()
    assert want.abs().max() < 2 ** 21  # in steps of a quarter: 23 bits
    assert got is out.view and torch.equal(got.cpu(), ref.rounded(want, t))
    out.check()
    b = torch.full((N + 8,), float("nan"), dtype=t, device="cuda")
    b[:N] = bias.to(t).cuda()
    got = ttc.gemm_w4(xd, w.w, b[:N], "relu")
    assert torch.equal(got.cpu(), ref.rounded(ref.act(want + bias, "relu"), t))


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (4, 1000, 700), (7, 129, 4096), (16, 500, 333),
                                   (30, 200, 1030), (64, 300, 2000)])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_w4_random(M, N, K, name, dtype):
    t = DTYPES[dtype]
    g = gen("w4 random", M, N, K, name, dtype)
    x = normal(g, t, M, K, std=4.0 / K ** 0.5)
    for group, zeros in ((32, True), (64, False), (128, True)):
        w = W4(g, N, K, group, zeros, t)
        bias = normal(g, t, N)
        y = ttc.gemm_w4(dev(x, t), w.w, bias.to(t).cuda(), name)
        ref.close(y, *ref.w4_bound(x, w.value, bias, name, t), f"{M} x {N} x {K} {name} {group}")


@pytest.mark.parametrize("M,F,D", W4_SIZES)
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_w4_gated(M, F, D, group, zeros, dtype):
    t = DTYPES[dtype]
    g = gen("w4 gated", M, F, D, group, zeros)
    x = integers(g, -1, 1, M, D)
    wg, wu = (W4(g, F, D, group, zeros, t, exact=True) for _ in range(2))
    for name in ("none", "relu"):
        out = Out(M, F, t)
        got = ttc.gemm_gated_w4(dev(x, t, 8, 1), wg.w, wu.w, name, out.view)
        gate, up = x @ wg.value.t(), x @ wu.value.t()
        # gate and up are exact, their product is one fp32 multiplication
        want = (ref.act(gate, name).float() * up.float()).to(t)
        assert torch.equal(got.cpu(), want)
        out.check()
    x = normal(g, t, M, D, std=4.0 / D ** 0.5)
    wg, wu = (W4(g, F, D, group, zeros, t) for _ in range(2))
    for name in ("silu", "gelu"):
        r = ref.Gated(x, wg.value, wu.value, name)
        ref.close(ttc.gemm_gated_w4(dev(x, t), wg.w, wu.w, name), r.h, r.h_bound(t), name)


@pytest.mark.parametrize("dtype", DTYPES)
def test_w4_every_code_and_zero(dtype):
    """All 16 codes with all 16 zero points in every place of a word."""
    t = DTYPES[dtype]
    K = 256
    codes = torch.arange(16)[:, None].expand(16, K).repeat(16, 1)
    zeros = torch.arange(16).repeat_interleave(16)[None].expand(K // 32, 256)
    w = ttc.w4_pack(codes.to(torch.uint8).cuda(), torch.ones(256, K // 32, dtype=t, device="cuda"),
                    zeros.t().to(torch.uint8).contiguous().cuda(), group=32)
    assert torch.equal(ttc.w4_unpack(w).cpu().long(), codes)
    want = ref.weight(codes, torch.ones(K // 32, 256), zeros, 32)
    for start in range(0, K, 64):
        x = torch.zeros(64, K, dtype=torch.float64)
        x[torch.arange(64), torch.arange(64) + start] = 1
        got = ttc.gemm_w4(dev(x, t), w)
        assert torch.equal(got.cpu().double(), want[:, start:start + 64].t())


@pytest.mark.parametrize("M", [1, 20, 64])
@pytest.mark.parametrize("dtype", DTYPES)
def test_w4_special_values(M, dtype):
    """A scale that is NaN or infinite reaches its output column alone; NaN in x its row."""
    t = DTYPES[dtype]
    g = gen("w4 special", M)
    N, K = 200, 500
    x = normal(g, t, M, K)
    w = W4(g, N, K, 64, True, t)
    base = ttc.gemm_w4(dev(x, t), w.w).cpu()
    scales = w.w.scales.clone()
    keep = torch.ones(N, dtype=torch.bool)
    keep[[3, 130]] = False
    w.w.scales[2, 3], w.w.scales[7, 130] = float("nan"), float("inf")
    got = ttc.gemm_w4(dev(x, t), w.w).cpu()
    assert torch.equal(got[:, keep], base[:, keep])
    assert not got[:, 3].isfinite().any() and not got[:, 130].isfinite().any()
    w.w.scales.copy_(scales)
    x2 = x.clone()
    x2[M - 1, K - 1] = float("nan")
    got = ttc.gemm_w4(dev(x2, t), w.w).cpu()
    assert got[M - 1].isnan().all() and torch.equal(got[:M - 1], base[:M - 1])


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [1, 4, 8, 9, 64])
@pytest.mark.parametrize("dtype", DTYPES)
def test_w4_infinities(M, zeros, dtype):
    """Infinities in x: what their codes make of them, in their rows alone."""
    t = DTYPES[dtype]
    g = gen("w4 infinities", M, zeros)
    N, K = 77, 600
    x = normal(g, t, M, K)
    w, u = (W4(g, N, K, 64, zeros, t) for _ in range(2))
    base = ttc.gemm_w4(dev(x, t), w.w).cpu()
    x[M - 1, 130] = float("inf")
    want = x[M - 1:] @ w.value.t()  # +-infinity, NaN where the weight is 0
    got = ttc.gemm_w4(dev(x, t), w.w).cpu()
    assert torch.equal(got[:M - 1], base[:M - 1])
    assert torch.equal(got[M - 1:].double().nan_to_num(7.0), want.nan_to_num(7.0))
    assert want.isinf().any()
    want = want.clamp(min=0).nan_to_num(0.0, posinf=float("inf")) * (x[M - 1:] @ u.value.t())  # ReLU of NaN: 0
    got = ttc.gemm_gated_w4(dev(x, t), w.w, u.w, "relu").cpu()[M - 1:].double()
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[got.isinf()], want[want.isinf()])
    x[M - 1, 131] = float("nan")
    assert ttc.gemm_w4(dev(x, t), w.w).cpu()[M - 1].isnan().all()


@pytest.mark.parametrize("M,N,K", [(1, 20000, 300), (8, 30011, 264), (3, 2400, 9000),
                                   (8, 40000, 4104)])
def test_w4_many_tiles(M, N, K):
    """More tiles than SMs, and than a CTA holds sums of at a time."""
    t = torch.bfloat16
    g = gen("tiles", M, N, K)
    w = W4(g, N, K, 128, True, t)
    x = integers(g, -1, 1, M, K)
    bias = integers(g, -8, 8, N)
    got = ttc.gemm_w4(dev(x, t), w.w, bias.to(t).cuda())
    ref.close(got, *ref.w4_bound(x, w.value, bias, "none", t))


@pytest.mark.parametrize("M", [1, 8])
@pytest.mark.parametrize("dtype", DTYPES)
def test_w4_range_of_x(M, dtype):
    """Groups of x at both ends of the type's range, and with values far apart."""
    t = DTYPES[dtype]
    g = gen("range", M)
    N, K = 40, 512
    # (bf16: as far as sums and what they are rounded to stay normal numbers)
    lo, hi = (-14, 10) if t is torch.float16 else (-90, 90)
    x = normal(g, t, M, K) * 2.0 ** torch.randint(lo, hi, (M, K // 32), generator=g).double() \
        .repeat_interleave(32, 1)
    x = x.to(t).double()
    w = W4(g, N, K, 32, True, t)
    # codes and zero points may be summed apart: magnitudes count both
    both = ref.weight(w.codes, w.scales.abs(), -w.zeros, 32)
    for group in range(K // 32):
        part = torch.zeros_like(x)
        at = slice(32 * group, 32 * group + 32)
        part[:, at] = x[:, at]
        for y in (part, x) if group == 0 else (part,):
            want, r = y @ w.value.t(), ref.HALF[t]
            off = ref.sum_bound(32 if y is part else K, y.abs() @ both.t())
            ref.close(ttc.gemm_w4(dev(y, t), w.w), want,
                      off * (1 + r) + r * want.abs() + ref.TINY[t])


@pytest.mark.parametrize("M", [1, 5, 8])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_small_bf16_results(M, group):
    """Few rows whose results go down to bf16's subnormals keep bf16's bits."""
    t = torch.bfloat16
    g = gen("small", M, group)
    N, K = 70, 512
    w = W4(g, N, K, group, True, t)
    both = ref.weight(w.codes, w.scales.abs(), -w.zeros, group)
    for exponent in (-104, -110, -116, -122, -128):
        x = (torch.randn(M, K, generator=g).double() * 2.0 ** exponent).to(t).double()
        want, r = x @ w.value.t(), ref.HALF[t]
        # fp32 results below 2^-126 are off by up to 2^-150 each: 3 for each of up to 16 groups and
        # 16 more for joining them, all in terms of the result or of it by a scale below 1
        assert w.scales.abs().max() < 1
        off = ref.sum_bound(K, x.abs() @ both.t()) + 64 * 2.0 ** -150
        ref.close(ttc.gemm_w4(dev(x, t), w.w), want, off * (1 + r) + r * want.abs() + ref.TINY[t],
                  f"2^{exponent}")


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [1, 8])
@pytest.mark.parametrize("group", [32, 128])
def test_w4_large_bf16_values(M, group, zeros):
    """Values of x close to bf16's largest, in their rows alone; a code at its zero point takes
    them out of a result."""
    t = torch.bfloat16
    g = gen("large", M, group, zeros)
    N, K = 90, 400
    x = normal(g, t, M, K)
    w = W4(g, N, K, group, zeros, t)
    base = ttc.gemm_w4(dev(x, t), w.w).cpu()
    for exponent in (115, 116, 119, 122):
        x[M - 1, 133] = 2.0 ** exponent
        want, r = x @ w.value.t(), ref.HALF[t]
        assert want.abs().max() < 2.0 ** 127
        got = ttc.gemm_w4(dev(x, t), w.w).cpu()
        assert torch.equal(got[:M - 1], base[:M - 1])
        # summed in one chain of fp32 additions a group, then one of the groups (from 2^116 on; below,
        # codes and zero points apart, to which a code at its zero point is no exception)
        if exponent >= 116:
            off = (group + -(-K // group)) * 2.0 ** -24 * (x.abs() @ w.value.abs().t())
        else:
            both = ref.weight(w.codes, w.scales.abs(), -w.zeros if zeros else
                              torch.full(w.scales.shape, -8), group)
            off = ref.sum_bound(K, x.abs() @ both.t())
            # x is held to 2^-35 of the largest value of its group
            at = slice(133 // group * group, 133 // group * group + group)
            steps = w.codes[:, at].double().sum(1) * w.scales[133 // group].abs()
            off[M - 1] += 2.0 ** (exponent - 35) * steps
        ref.close(got[M - 1:], want[M - 1:],
                  (off * (1 + r) + r * want.abs() + ref.TINY[t])[M - 1:], f"2^{exponent}")
    # (a column whose code is its zero point was among them)
    assert exponent >= 116 and (want[M - 1].abs() < 2.0 ** 20).any()


@pytest.mark.parametrize("M", [1, 8])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_large_bf16_sums(M, group):
    """Sums of a group that pass bf16's and fp32's largest value, and results that do not."""
    t = torch.bfloat16
    N, K = 40, 256
    codes = torch.full((N, K), 15, dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // group), 2.0 ** -12, dtype=t, device="cuda")
    for zero, factor in ((0, 15 / 16), (7, 1 / 2), (None, 7 / 16)):
        zeros = None if zero is None else torch.full((N, K // group), zero, dtype=torch.uint8,
                                                     device="cuda")
        w = ttc.w4_pack(codes, scales, zeros, group=group)
        for exponent in (114, 115, 116, 117, 120, 126, 127):
            for mantissa in (1.0, 1.25, 1.9921875):
                x = torch.full((M, K), mantissa * 2.0 ** exponent, dtype=t, device="cuda")
                want = torch.tensor(mantissa * 2.0 ** exponent * factor).to(t)
                assert (ttc.gemm_w4(x, w).cpu() == want).all(), (zero, exponent, mantissa)


def test_w4_slices_of_rows():
    """Rows of a weight are a weight."""
    t = torch.float16
    g = gen("slices")
    w = W4(g, 400, 600, 32, True, t)
    x = normal(g, t, 12, 600)
    for a, b in ((0, 128), (16, 400), (160, 333)):
        part = ttc.W4Tensor(w.w.data[a:b], w.w.scales[:, a:b], w.w.zeros[:, a:b], b - a, 600, 32)
        ref.close(ttc.gemm_w4(dev(x, t), part), *ref.w4_bound(x, w.value[a:b], None, "none", t))


# ------------------------------------------------------- long sums, many tiles, few rows ---
#
# Sizes at which the kernels' rings of shared memory are gone through more than once (rings of
# up to 7 places of 64 columns, 12 for the fewest rows; of up to 6 of 256 for 4 bits), K
# divided and not, one wave of tiles and more.  References are 64-bit products on the GPU.

SPLIT = [(250, 4096),   # F, D: few tiles, K in several parts of 8 blocks or more
         (4700, 4096),  # 74 tiles
         (6000, 1024),  # 94: one a CTA with the deep ring
         (10300, 640)]  # 161: more than SMs


@pytest.mark.parametrize("F,D", SPLIT)
@pytest.mark.parametrize("M", [1, 4, 16, 30, 60, 100])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_long_sums(M, F, D, dtype):
    t = DTYPES[dtype]
    g = gen("long", M, F, D)
    x, wg, wu = (integers(g, -1, 1, *s).cuda() for s in ((M, D), (F, D), (F, D)))
    h, gate, up = ttc.gemm_gated(x.to(t), wg.to(t), wu.to(t), "relu", save=True)
    a, b = x @ wg.t(), x @ wu.t()
    assert torch.equal(gate.double(), a) and torch.equal(up.double(), b)
    assert torch.equal(h, ref.rounded(a.clamp(min=0) * b, t))


@pytest.mark.parametrize("F,D", [(2000, 256),    # two tiles, K in several parts
                                 (520, 10000),   # 79: the deep ring
                                 (264, 19200)])  # 150: more than SMs
@pytest.mark.parametrize("M", [1, 4, 16, 30, 60, 100])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_backward_long_sums(M, F, D, dtype):
    t = DTYPES[dtype]
    backward_exact(t, gen("long backward", M, F, D), M, F, D)


def backward_exact(t, g, M, F, D):
    """Gradients of small integers, whose roundings to 16 bits and sums are exact."""
    # gates and ups stay small: so many of x are 0 that a sum of D products, of which 4 in 9
    # count otherwise, has a deviation of 3
    x = integers(g, -1, 1, M, D) * (torch.rand((M, D), generator=g) < 9 / (D * 4 / 9))
    x, wg, wu = (v.cuda() for v in (x, integers(g, -1, 1, F, D), integers(g, -1, 1, F, D)))
    dh = integers(g, -2, 2, M, F).cuda()
    r = ref.Gated(x, wg, wu, "relu")
    want = r.backward(dh, t)
    assert max(r.dg.abs().max(), r.du.abs().max()) <= 256
    args = x.to(t), wg.to(t), wu.to(t)
    _, gate, up = ttc.gemm_gated(*args, "relu", save=True)
    got = ttc.gemm_gated_backward(dh.to(t), *args, gate, up, "relu")
    for v, (k, (w, _)) in zip(got, want.items()):
        assert torch.equal(v, ref.rounded(w, t)), k


# dX on the kernel of large products: 48 tiles; 99, the second wave of which goes down K.  F is
# no multiple of 64: the seam between the two pairs of operands lies inside a block.
LARGE_DX = [(2000, 200, 1296), (2600, 136, 2104)]


@pytest.mark.parametrize("M,F,D", LARGE_DX)
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_backward_large_dx_exact(M, F, D, dtype):
    t = DTYPES[dtype]
    backward_exact(t, gen("large dx", M, F, D), M, F, D)


@pytest.mark.parametrize("M,F,D", LARGE_DX + [(2000, 203, 1290), (2600, 139, 2101)])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_backward_large_dx_random(M, F, D, name, dtype):
    t = DTYPES[dtype]
    g = gen("large dx", M, F, D, name, dtype)
    x = normal(g, t, M, D, std=2.0).cuda()
    wg, wu = (normal(g, t, F, D, std=2.0 / D ** 0.5).cuda() for _ in range(2))
    dh = normal(g, t, M, F, std=0.3).cuda()
    r = ref.Gated(x, wg, wu, name)
    args = dev(x, t), dev(wg, t), dev(wu, t)
    _, gate, up = ttc.gemm_gated(*args, name, save=True)
    got = ttc.gemm_gated_backward(dev(dh, t), *args, gate, up, name)
    for v, (k, (w, bound)) in zip(got, r.backward(dh, t).items()):
        ref.close(v, w.cpu(), bound.cpu(), f"{k} {M} x {F} x {D} {name}")


def w4_on_gpu(g, rows, cols, group, zeros, t):
    """A weight with scales of powers of two, and its 64-bit values."""
    groups = -(-cols // group)
    codes = torch.randint(0, 16, (rows, cols), generator=g, dtype=torch.uint8).cuda()
    scales = torch.exp2(torch.randint(-4, 0, (rows, groups), generator=g).double()).cuda()
    z = torch.randint(0, 16, (rows, groups), generator=g, dtype=torch.uint8).cuda() if zeros else None
    w = ttc.w4_pack(codes, scales.to(t), z, group=group)
    at = torch.arange(cols, device="cuda") // group
    value = codes.double() - (z.double()[:, at] if zeros else 8.0)
    return w, value.mul_(scales[:, at])


@pytest.mark.parametrize("M,N,K", [(1, 200, 16384), (4, 200, 32768), (8, 200, 16384),  # K > N
                                   (13, 200, 16384), (30, 200, 16384), (61, 200, 16384),
                                   (130, 200, 16384), (16, 70, 9000),
                                   # one part; tiles for more than a wave
                                   (16, 38000, 2600), (32, 38000, 2600), (64, 38000, 2600)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", DTYPES)
def test_w4_long_sums(M, N, K, group, dtype):
    """Sums are exact: at most 32768 products of 7.5 in steps of a sixteenth, 22 bits."""
    t = DTYPES[dtype]
    g = gen("w4 long", M, N, K, group)
    x = integers(g, -1, 1, M, K).cuda()
    w, value = w4_on_gpu(g, N, K, group, group != 64, t)
    want = x @ value.t()
    assert torch.equal(ttc.gemm_w4(dev(x, t), w), ref.rounded(want, t))
    # gated: the first and the last rows of the weight (a slice starts on 16 rows)
    first, F = N // 2 // 16 * 16, N - N // 2 // 16 * 16

    def part(a, b):
        z = None if w.zeros is None else w.zeros[:, a:b]
        return ttc.W4Tensor(w.data[a:b], w.scales[:, a:b], z, b - a, K, group)

    got = ttc.gemm_gated_w4(dev(x, t), part(0, F), part(first, N), "relu")
    gate, up = want[:, :F].float(), want[:, first:].float()
    assert torch.equal(got, (gate.clamp(min=0) * up).to(t))


# --------------------------------------------------------------- empty, use, refusals ---


@pytest.mark.parametrize("dtype", DTYPES)
def test_empty(dtype):
    t = DTYPES[dtype]

    def m(r, c, v=1.0, kind=t):
        return torch.full((r, c), v, dtype=kind, device="cuda")

    for M, F, D in [(0, 5, 8), (5, 0, 8), (5, 16, 0), (0, 0, 0)]:
        h, gate, up = ttc.gemm_gated(m(M, D), m(F, D), m(F, D), save=True)
        assert h.shape == (M, F) and (h == 0).all() and (gate == 0).all() and (up == 0).all()
        dx, dwg, dwu = ttc.gemm_gated_backward(m(M, F), m(M, D), m(F, D), m(F, D), gate, up)
        assert dx.shape == (M, D) and dwg.shape == dwu.shape == (F, D)
        assert (dx == 0).all() and (dwg == 0).all() and (dwu == 0).all()
    for M, N, K in [(0, 16, 64), (3, 0, 64), (3, 16, 0)]:
        groups = -(-K // 64)
        w = ttc.W4Tensor(torch.zeros(N, -(-K // 32) * 16, dtype=torch.uint8, device="cuda"),
                         m(groups, N), None, N, K, 64)
        bias = torch.arange(N, device="cuda").to(t)
        assert torch.equal(ttc.gemm_w4(m(M, K), w, bias), bias.expand(M, N))
        assert (ttc.gemm_gated_w4(m(M, K), w, w) == 0).all()


def step(x, wg, wu, dh, w4a, w4b):
    h, gate, up = ttc.gemm_gated(x, wg, wu, "silu", save=True)
    grads = ttc.gemm_gated_backward(dh, x, wg, wu, gate, up, "silu")
    y = ttc.gemm_gated_w4(x[:5], w4a, w4b, "gelu")
    z = ttc.gemm_w4(x[:20], w4a, None, "relu")
    return (h, gate, up, *grads, y, z)


def step_inputs(seed, M=100, F=520, D=264):
    t = torch.bfloat16
    g = gen("step", seed)
    x, wg, wu, dh = (dev(normal(g, t, *s), t) for s in ((M, D), (F, D), (F, D), (M, F)))
    return x, wg, wu, dh, W4(g, F, D, 64, True, t).w, W4(g, F, D, 64, True, t).w


def test_same_bits_every_time():
    args = step_inputs(1)
    first = step(*args)
    for _ in range(5):
        for a, b in zip(first, step(*args)):
            assert torch.equal(a, b)


def test_streams_and_given_outputs():
    """Two streams at once, one of them passed by hand; new memory belongs to the call's stream."""
    one, two = step_inputs(1), step_inputs(2)
    want = [step(*one), step(*two)]
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(sa):
            a = step(*one)
        with torch.cuda.stream(sb):
            b = step(*two)
        c = ttc.gemm_gated(*one[:3], stream=sa)
        d = ttc.gemm_w4(one[0][:20], one[4], None, "relu", stream=sb)
        torch.cuda.synchronize()
        for got, w in ((a, want[0]), (b, want[1])):
            assert all(torch.equal(p, q) for p, q in zip(got, w))
        assert torch.equal(c, want[0][0]) and torch.equal(d, want[0][7])


def test_threads():
    args = [step_inputs(i) for i in range(4)]
    want = [step(*a) for a in args]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = step(*args[i])
                s.synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, want[i])):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_graphs():
    """Two captured graphs of all operators replayed in turn with new inputs."""
    sets = [step_inputs(i) for i in (1, 2)]
    other = [step_inputs(i) for i in (3, 4)]
    [step(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(*s))
        graphs.append(graph)
    for values in (sets, other, sets):
        values = [[(v if isinstance(v, torch.Tensor) else v.data).clone() for v in s] for s in values]
        for s, v in zip(sets, values):
            for a, b in zip(s, v):
                (a if isinstance(a, torch.Tensor) else a.data).copy_(b)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        got = [[o.clone() for o in out] for out in outs]
        for s, out in zip(sets, got):
            assert all(torch.equal(p, q) for p, q in zip(out, step(*s)))


def test_layer_with_the_other_operators():
    """A block as it is served: norm, gated projections in 16 bits and in 4, down projection."""
    t = torch.float16
    g = gen("layer")
    M, D, F = 9, 256, 768
    x, res = normal(g, t, M, D), normal(g, t, M, D)
    gain, down = 1 + normal(g, t, D, std=0.1), normal(g, t, F, D, std=F ** -0.5)
    y, h = ttc.rms_norm(dev(x, t), gain.to(t).cuda(), residual=dev(res, t))
    for four_bits in (False, True):
        if four_bits:
            a, b = (W4(g, F, D, 128, True, t) for _ in range(2))
            got = ttc.gemm_gated_w4(y, a.w, b.w)
            wg, wu = a.value, b.value
        else:
            wg, wu = (normal(g, t, F, D, std=D ** -0.5) for _ in range(2))
            got = ttc.gemm_gated(y, dev(wg, t), dev(wu, t))
        r = ref.Gated(y.cpu().double(), wg, wu, "silu")
        ref.close(got, r.h, r.h_bound(t))
        out = ttc.gemm_f16(got, dev(down, t))
        want = got.cpu().double() @ down
        ref.close(out, want, ref.sum_bound(F, got.cpu().double().abs() @ down.abs()) +
                  ref.HALF[t] * want.abs() + 1e-6)


def test_far_rows():
    """Rows and outputs past 2^31 bytes and 2^31 elements from the start."""
    t = torch.float16
    M, F, D = 5, 40, 64
    g = gen("far")
    x, wg, wu = (normal(g, t, *s) for s in ((M, D), (F, D), (F, D)))
    r = ref.Gated(x, wg, wu, "silu")
    ld = (1 << 30) + 64  # the fifth row starts past 2^32 elements
    big = torch.empty(4 * ld + (1 << 22), dtype=t, device="cuda")
    xs = big.as_strided((M, D), (ld, 1))
    xs.copy_(x.to(t))
    hs = big.as_strided((M, F), (ld, 1), 1 << 20)
    hs = ttc.gemm_gated(xs, dev(wg, t), dev(wu, t), out=hs)
    ref.close(hs, r.h, r.h_bound(t))
    w = W4(g, F, D, 32, True, t)
    ys = big.as_strided((M, F), (ld, 1), 1 << 21)
    ttc.gemm_w4(xs, w.w, out=ys)
    ref.close(ys, *ref.w4_bound(x, w.value, None, "none", t))


def test_refusals():
    t = torch.float16
    x, w = torch.zeros(4, 64, dtype=t, device="cuda"), torch.zeros(16, 64, dtype=t, device="cuda")
    h = torch.zeros(4, 16, dtype=t, device="cuda")
    f = torch.zeros(4, 16, device="cuda")
    with pytest.raises(ValueError, match="act"):
        ttc.gemm_gated(x, w, w, "tanh")
    with pytest.raises(RuntimeError):
        ttc.gemm_gated(x, w, w, 4)
    for bad in [(x.float(), w, w), (x, w.bfloat16(), w), (x, w, w.float())]:
        with pytest.raises(TypeError):
            ttc.gemm_gated(*bad)
    for bad in [(x[0], w, w), (x, w[:, :32], w), (x, w, w[:8]), (x.cpu(), w, w), (x, w.cpu(), w),
                (x.t().contiguous().t(), w, w)]:
        with pytest.raises(ValueError):
            ttc.gemm_gated(*bad)
    odd = torch.zeros(4 * 65 + 8, dtype=t, device="cuda")
    for bad in (odd[:4 * 65].view(4, 65)[:, :64], odd[1:257].view(4, 64)):  # stride, address
        with pytest.raises(RuntimeError, match="align"):
            ttc.gemm_gated(bad, w, w)
    with pytest.raises(RuntimeError):  # rows that overlap
        ttc.gemm_gated(x[:1].expand(4, 64), w, w)
    with pytest.raises(RuntimeError):  # an output that is an input
        ttc.gemm_gated(x[:, :16], w[:, :16], w[:, :16], out=x[:, :16])
    with pytest.raises(TypeError):
        ttc.gemm_gated_backward(h, x, w, w, h, h)
    with pytest.raises(ValueError):
        ttc.gemm_gated_backward(h, x, w, w, f[:, :8], f)
    with pytest.raises(ValueError):
        ttc.gemm_gated_backward(h[:3], x, w, w, f, f)
    q = ttc.w4_pack(torch.zeros(16, 64, dtype=torch.uint8, device="cuda"),
                    torch.ones(16, 1, dtype=t, device="cuda"), group=64)
    with pytest.raises(TypeError):
        ttc.gemm_w4(x.bfloat16(), q)
    with pytest.raises(ValueError):
        ttc.gemm_w4(x[:, :32], q)
    with pytest.raises(ValueError):
        ttc.gemm_w4(x, q, bias=torch.zeros(15, dtype=t, device="cuda"))
    with pytest.raises(ValueError):
        ttc.gemm_w4(x, q, out=h[:, :15])
    with pytest.raises(RuntimeError):
        ttc.gemm_w4(x, q, act=9)
    z = ttc.W4Tensor(q.data, q.scales, torch.zeros(1, 16, dtype=torch.uint8, device="cuda"), 16, 64,
                     64)
    with pytest.raises(ValueError):
        ttc.gemm_gated_w4(x, q, z)
    assert (ttc.gemm_w4(x, q) == 0).all() and ttc.ff_device_status() == 0


def test_codes_past_32_bits():
    """An activation's code that no int holds is refused, not cut to one that exists."""
    t = torch.float16
    x, w = torch.zeros(4, 64, dtype=t, device="cuda"), torch.zeros(16, 64, dtype=t, device="cuda")
    h, f = torch.zeros(4, 16, dtype=t, device="cuda"), torch.zeros(4, 16, device="cuda")
    q = ttc.w4_pack(torch.zeros(16, 64, dtype=torch.uint8, device="cuda"),
                    torch.ones(16, 1, dtype=t, device="cuda"), group=64)
    m = ttc.mx_quantize(x, "mxfp8")
    for act in (1 << 32, (1 << 32) + 3, -(1 << 32)):
        for call in (lambda: ttc.gemm_gated(x, w, w, act), lambda: ttc.gemm_w4(x, q, act=act),
                     lambda: ttc.gemm_gated_backward(h, x, w, w, f, f, act),
                     lambda: ttc.gemm_gated_w4(x, q, q, act),
                     lambda: ttc.gemm_mx(m, m, None, act)):
            with pytest.raises(RuntimeError):
                call()
    with pytest.raises(OverflowError):
        ttc.gemm_gated(x, w, w, 1 << 64)


def test_gradients_are_not_lost_in_silence():
    """A backward pass through a result without a graph raises; calls without one are as before."""
    t = torch.float16
    g = gen("no graph")
    x, wg, wu = (dev(normal(g, t, *s), t) for s in ((4, 64), (16, 64), (16, 64)))
    w = W4(g, 16, 64, 64, False, t).w
    b = torch.ones(16, dtype=t, device="cuda")
    h, y, z = ttc.gemm_gated(x, wg, wu), ttc.gemm_w4(x, w, b), ttc.gemm_gated_w4(x, w, w)
    assert not (h.requires_grad or y.requires_grad or z.requires_grad)

    def leaf(v):
        return v.detach().requires_grad_()

    learned = ttc.W4Tensor(w.data, leaf(w.scales), None, 16, 64, 64)  # (its scales)
    calls = [(h, lambda **k: ttc.gemm_gated(leaf(x), wg, wu, **k), "gemm_gated_backward"),
             (h, lambda **k: ttc.gemm_gated(x, leaf(wg), wu, **k), "gemm_gated_backward"),
             (h, lambda **k: ttc.gemm_gated(x, wg, leaf(wu), **k), "gemm_gated_backward"),
             (y, lambda **k: ttc.gemm_w4(leaf(x), w, b, **k), "gemm_w4 has no"),
             (y, lambda **k: ttc.gemm_w4(x, w, leaf(b), **k), "gemm_w4 has no"),
             (y, lambda **k: ttc.gemm_w4(x, learned, b, **k), "gemm_w4 has no"),
             (z, lambda **k: ttc.gemm_gated_w4(leaf(x), w, w, **k), "gemm_gated_w4 has no"),
             (z, lambda **k: ttc.gemm_gated_w4(x, w, learned, **k), "gemm_gated_w4 has no")]
    for want, call, message in calls:
        got = call()
        assert torch.equal(got.detach(), want) and got.requires_grad
        with pytest.raises(RuntimeError, match=message):
            got.float().sum().backward()
        out = torch.zeros_like(want)
        with pytest.raises(RuntimeError, match=message):
            call(out=out)
        assert (out == 0).all()
        with torch.no_grad():
            assert call(out=out) is out and torch.equal(out, want)
            assert not call().requires_grad
    # nor is it handed out as None, and a kept result holds nothing of the inputs' gradients
    v = leaf(x)
    got = ttc.gemm_gated(v, wg, wu)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(got.float().sum(), v)
    assert got.grad_fn.next_functions == ()
    # with save the gradients are the caller's own business
    results = ttc.gemm_gated(leaf(x), leaf(wg), leaf(wu), save=True)
    assert torch.equal(results[0], h) and not any(v.requires_grad for v in results)
    results[0].requires_grad_().float().sum().backward()
    grads = ttc.gemm_gated_backward(results[0].grad, leaf(x), leaf(wg), leaf(wu), *results[1:])
    assert not any(v.requires_grad for v in grads)


def test_library_refuses_what_the_binding_cannot_see():
    """Through the C boundary: extents past the allocation, host pointers, too large strides."""
    import ctypes
    lib = ttc.ff_lib()
    x = torch.zeros(1 << 20, dtype=torch.float16, device="cuda")
    p, n = ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(0)
    o = ctypes.c_void_p(x.data_ptr() + (1 << 20))
    host = ctypes.c_void_p(torch.zeros(4096, dtype=torch.float16).data_ptr() & ~15)

    def gated(X, Wg, Wu, H, M=4, F=16, D=64, ld=64, ldh=16, G=n, U=n):
        return lib.ff_gated(X, Wg, Wu, H, G, U, M, F, D, ld, ld, ld, ldh, 16, 16, 0, 3, None)

    assert gated(p, p, p, o) == 0
    assert gated(host, p, p, o) == -1 and gated(p, p, p, host) == -1 and gated(n, p, p, o) == -1
    # (137 GB of rows: more than any segment that the allocator may have put x into)
    assert gated(p, p, p, o, M=1 << 30) == -1 and gated(p, p, p, o, ld=60) == -1
    assert gated(p, p, p, o, ld=68) == -2 and gated(p, p, p, o, ldh=1 << 40) == -1
    assert gated(p, p, p, o, M=(1 << 31) - 300, ld=1 << 38) == -1  # wraps in 64 bits
    assert gated(p, p, p, o, G=ctypes.c_void_p(x.data_ptr() + (1 << 19))) == -1  # gate without up
    assert gated(p, p, p, p) == -1
    torch.cuda.synchronize()
    assert ttc.ff_device_status() == 0
