"""What the microscaled operators do without a GPU: the boundary as a C consumer
sees it, refusals before any device work, the storage layout, and the plain
implementation the GPU tests rely on, against things other than itself."""
import ctypes
import math
import os
import re
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

import mx_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_mx.h")


@pytest.fixture(scope="module")
def ttc():
    import tiled_tensor_core_05_b200 as pkg
    from tiled_tensor_core_05_b200 import build
    build.build()
    pkg.mx_lib()
    return pkg


def declared():
    return re.findall(r"GEMM_API\s+[\w\s\*]+?\b(mx_\w+)\s*\(", open(HEADER).read())


def test_exports_are_the_declared_functions(ttc):
    from tiled_tensor_core_05_b200 import mx
    out = subprocess.run(["nm", "-D", "--defined-only", mx.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines()
                if line.split() and line.split()[-2] in ("T", "W")}
    assert exported == set(declared())
    assert set(mx._SIGNATURES) == set(declared())


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_c_consumer(ttc, tmp_path):
    from tiled_tensor_core_05_b200 import mx
    src = tmp_path / "use.c"
    src.write_text('#include <stdio.h>\n#include "gemm_mx.h"\ntypedef void (*fn)(void);\n'
                   "int main(void) {\n  const fn f[] = {" +
                   ", ".join(f"(fn){n}" for n in declared()) + "};\n"
                   '  printf("%d %d %d\\n", (int)(sizeof(f) / sizeof(f[0])), mx_abi_version(),\n'
                   "         mx_quantize(0, 0, 0, -1, 1, 8, 16, MX_F16, MX_FP4, 0));\n"
                   "  return f[0] == 0;\n}\n")
    exe = tmp_path / "use"
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe), mx.LIB_PATH,
                    f"-Wl,-rpath,{os.path.dirname(mx.LIB_PATH)}"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out == [str(len(declared())), "10000", "-1"]


def test_refusals_before_device_work(ttc):
    lib = ttc.mx_lib()
    n = ctypes.c_void_p(0)
    big = 1 << 31
    for rows, cols, dtype, fmt in [(-1, 4, 0, 1), (4, -1, 0, 1), (big, 4, 0, 1), (4, big, 0, 1),
                                   (4, 4, 2, 1), (4, 4, -1, 1), (4, 4, 0, 0), (4, 4, 0, 3)]:
        assert lib.mx_quantize(n, n, n, rows, cols, 8, 16, dtype, fmt, None) == -1
        assert lib.mx_dequantize(n, n, n, rows, cols, 16, 8, dtype, fmt, None) == -1
        if fmt != 0:
            assert lib.mx_rms_norm(n, n, n, n, n, n, rows, cols, 8, 8, 8, 16, 1e-6, dtype, fmt,
                                   None) == -1
    for eps in (-1e-6, math.nan):
        assert lib.mx_rms_norm(n, n, n, n, n, n, 4, 4, 8, 8, 8, 16, eps, 0, 0, None) == -1
    one = ctypes.c_void_p(16)
    # a residual output without a residual
    assert lib.mx_rms_norm(n, n, n, one, n, n, 0, 4, 8, 8, 8, 16, 1e-6, 0, 0, None) == -1
    for M, N, K, fmt, dtype, act in [(-1, 4, 4, 1, 0, 0), (4, -1, 4, 1, 0, 0), (4, 4, -1, 1, 0, 0),
                                     (big, 4, 4, 1, 0, 0), (4, 4, big, 1, 0, 0), (4, 4, 4, 0, 0, 0),
                                     (4, 4, 4, 3, 0, 0), (4, 4, 4, 1, 2, 0), (4, 4, 4, 1, 0, 3),
                                     (4, 4, 4, 1, 0, -1)]:
        assert lib.mx_gemm(n, n, n, n, n, n, M, N, K, 16, 16, 8, fmt, dtype, act, None) == -1
    # nothing to do: whatever the pointers
    assert lib.mx_quantize(n, n, n, 0, 5, 8, 16, 0, 1, None) == 0
    assert lib.mx_dequantize(n, n, n, 5, 0, 16, 8, 1, 2, None) == 0
    assert lib.mx_rms_norm(n, n, n, n, n, n, 0, 5, 8, 8, 8, 16, 0.0, 0, 0, None) == 0
    assert lib.mx_gemm(n, n, n, n, n, n, 0, 5, 5, 16, 16, 8, 1, 0, 0, None) == 0
    assert lib.mx_gemm(n, n, n, n, n, n, 5, 0, 5, 16, 16, 8, 2, 1, 2, None) == 0


def test_sizes(ttc):
    lib = ttc.mx_lib()
    for rows, cols in [(0, 0), (1, 1), (128, 128), (129, 129), (1000, 4097), (28672, 8192)]:
        for fmt, code in (("mxfp8", 1), ("mxfp4", 2)):
            assert lib.mx_row_bytes(cols, code) == ttc.mx_row_bytes(cols, fmt) == \
                ref.row_bytes(cols, fmt)
        assert lib.mx_scale_bytes(rows, cols) == ttc.mx_scale_bytes(rows, cols)
    assert lib.mx_row_bytes(4, 0) == lib.mx_row_bytes(-1, 1) == lib.mx_scale_bytes(-1, 4) == -1


@pytest.mark.parametrize("rows,cols", [(1, 1), (31, 33), (128, 128), (129, 257), (300, 4096)])
def test_scale_layout(ttc, rows, cols):
    rng = np.random.default_rng(rows)
    s = rng.integers(1, 255, (rows, -(-cols // 32))).astype(np.uint8)
    tiled = ttc.mx_tile_scales(torch.from_numpy(s))
    assert tiled.numel() == ttc.mx_scale_bytes(rows, cols)
    assert np.array_equal(tiled.numpy(), ref.tile_scales(s, cols))
    assert np.array_equal(ttc.mx_untile_scales(tiled, rows, cols).numpy(), s)


def test_python_refusals(ttc):
    x = torch.zeros(4, 64, dtype=torch.float16)
    data, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    q = ttc.MxTensor(data, scales, 4, 64, "mxfp8")
    with pytest.raises(ValueError, match="CUDA"):
        ttc.mx_quantize(x, "mxfp8")
    with pytest.raises(ValueError, match="format"):
        ttc.mx_quantize(x, "fp8")
    with pytest.raises(TypeError):
        ttc.mx_quantize(x.float(), "mxfp8")
    with pytest.raises(ValueError):
        ttc.mx_dequantize(q)
    with pytest.raises(TypeError):
        ttc.mx_dequantize(data)
    with pytest.raises(TypeError):
        ttc.gemm_mx(x, q)
    with pytest.raises(TypeError):
        ttc.rms_norm(x.float(), x[0])
    for bad in [(data.float(), scales, 4, 64, "mxfp8"), (data, scales.int(), 4, 64, "mxfp8")]:
        with pytest.raises(TypeError):
            ttc.MxTensor(*bad)
    for bad in [(data, scales, 5, 64, "mxfp8"), (data, scales, 4, 65, "mxfp8"),
                (data, scales[:511], 4, 64, "mxfp8"), (data, scales, 4, 64, "mxfp6"),
                (data.t(), scales, 64, 4, "mxfp8"), (data[0], scales, 4, 64, "mxfp8"),
                (data, scales.view(2, 256), 4, 64, "mxfp8")]:
        with pytest.raises(ValueError):
            ttc.MxTensor(*bad)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_extents_past_64_bits(tmp_path):
    """The size of an operand and whether an allocation holds it, for the sizes and strides that
    the entry points admit: rows below 2^31, rows less than 2^40 bytes apart."""
    src = tmp_path / "extent.cc"
    src.write_text('#include <stdio.h>\n#include "extent.h"\nint main() {\n'
                   "  long long r, u, l, t; unsigned long long p, b, n;\n"
                   '  while (scanf("%lld %lld %lld %lld %llu %llu %llu", &r, &u, &l, &t, &p, &b, &n) '
                   "== 7) {\n    const uint64_t s = ttc::matrix_span(r, u, l, t);\n"
                   '    printf("%llu %d\\n", (unsigned long long)s, ttc::span_inside(p, s, b, n));\n'
                   "  }\n}\n")
    exe = tmp_path / "extent"
    csrc = os.path.join(ROOT, "tiled_tensor_core_05_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", csrc, str(src), "-o",
                    str(exe)], check=True)
    base, size = 1 << 40, 1 << 21
    operands = [(1, 64, 64, 2), (8, 64, 64, 1), (2 ** 25 + 1, 64, 2 ** 38, 2),
                (2 ** 24 + 1, 64, 2 ** 39, 2), (2 ** 25 + 1, 64, 2 ** 39, 1),
                (2 ** 31 - 1, 8, 2 ** 40 - 16, 1), (2 ** 31 - 1, 8, 2 ** 39 - 8, 2),
                (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 + 7, 2), (1, 2 ** 62, 2 ** 62, 4),
                (1, 2 ** 62 + 3, 2 ** 62 + 3, 4), (2 ** 24, 16, 2 ** 39, 2), (2 ** 24 + 1, 0, 2 ** 39, 2),
                (1, size // 2, size // 2, 2), (1, size // 2 + 1, size, 2)]
    rows = [(*o, base + at, base, size) for o in operands
            for at in (0, 16, size - 128, size - 16, size, size + 16, -16, 2 ** 63, 2 ** 64 - 2 ** 41)]
    rows = [(*r[:4], r[4] % 2 ** 64, *r[5:]) for r in rows]
    out = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, r)) for r in rows),
                         capture_output=True, text=True, check=True).stdout.split("\n")
    for (n, used, ld, unit, p, b, s), line in zip(rows, out):
        span = ((n - 1) * ld + used) * unit
        want = min(span, 2 ** 64 - 1)
        assert line == f"{want} {int(b <= p and p + span <= b + s)}", (n, used, ld, unit, p - b)


# ------------------------------------------------- the plain implementation itself ---


def test_magnitudes_are_the_types():
    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.magnitudes("mxfp8"), e4m3)
    assert ref.magnitudes("mxfp4").tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def test_nearest_against_casts_and_fractions():
    rng = np.random.default_rng(0)
    y = np.abs(rng.standard_normal(20000) * np.exp2(rng.integers(-12, 8, 20000))).astype(np.float32)
    y = y[y <= 448]
    v = ref.magnitudes("mxfp8")
    mids = (v[1:] + v[:-1]) / 2
    y = np.concatenate([y, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e3), v]).astype(np.float32)
    cast = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v[ref.nearest_codes(y.astype(np.float64), "mxfp8")], cast)
    v4 = [Fraction(v) for v in ref.magnitudes("mxfp4")]
    for z in np.arange(0, 8, 1 / 32):
        d = [abs(Fraction(z) - w) for w in v4]
        best = [i for i in range(8) if d[i] == min(d)]
        want = best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]
        assert ref.nearest_codes(np.array([z]), "mxfp4")[0] == want, z


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_quantize_definition(fmt):
    """Each block's scale is the largest power of two that keeps the maximum
    below 2^(emax + 1), and what comes back is within half a step or saturated."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 100)) * np.exp2(rng.integers(-20, 20, (50, 1)))
    codes, scales = ref.quantize(x, fmt)
    back = ref.values(codes, scales, fmt)
    largest = ref.magnitudes(fmt)[-1]
    for b in range(4):
        blk = slice(32 * b, min(100, 32 * b + 32))
        X = np.exp2(scales[:, b].astype(float) - 127)
        top = np.abs(x[:, blk]).max(1) / X
        assert ((top >= 2.0 ** ref.EMAX[fmt]) & (top < 2.0 ** (ref.EMAX[fmt] + 1))).all()
        y = np.clip(np.abs(x[:, blk]) / X[:, None], 0, largest)
        step = np.exp2(np.maximum(np.floor(np.log2(y)), 1 - (7 if fmt == "mxfp8" else 1))
                       - (3 if fmt == "mxfp8" else 1))
        assert (np.abs(np.abs(back[:, blk]) / X[:, None] - y) <= step / 2).all()
        assert (np.signbit(back[:, blk]) == np.signbit(x[:, blk])).all()
    codes, scales = ref.quantize(np.zeros((1, 32)), fmt)
    assert scales[0, 0] == 0 and not codes.any()
    x = np.ones((1, 64))
    x[0, 40] = np.nan
    codes, scales = ref.quantize(x, fmt)
    assert scales[0, 1] == 255 and scales[0, 0] != 255 and not codes[0, 32:].any()


def test_pack_and_round():
    c = np.arange(7, dtype=np.uint8)[None]
    assert ref.pack(c, "mxfp4").tolist() == [[0x10, 0x32, 0x54, 0x06]]
    assert np.array_equal(ref.unpack(ref.pack(c, "mxfp4"), 7, "mxfp4"), c)
    rng = np.random.default_rng(1)
    x = rng.standard_normal(10000) * np.exp2(rng.integers(-140, 126, 10000))
    x = x.astype(np.float32)  # fp32 values: torch's cast rounds once
    for t in (torch.float16, torch.bfloat16):
        want = torch.from_numpy(x).to(t).double().numpy()
        assert np.array_equal(ref.round_to(x.astype(np.float64), t), want)
