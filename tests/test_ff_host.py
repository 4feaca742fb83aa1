"""What the feed-forward operators do without a GPU: the boundary as a C consumer sees
it, refusals before any device work, the layout of 4-bit weights, and the plain
implementation the GPU tests rely on, against things other than itself."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import ff_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_ff.h")


@pytest.fixture(scope="module")
def ttc():
    import tiled_tensor_core_05_b200 as pkg
    from tiled_tensor_core_05_b200 import build
    build.build()
    pkg.ff_lib()
    return pkg


def declared():
    return re.findall(r"GEMM_API\s+[\w\s\*]+?\b(ff_\w+)\s*\(", open(HEADER).read())


def test_exports_are_the_declared_functions(ttc):
    from tiled_tensor_core_05_b200 import ff
    out = subprocess.run(["nm", "-D", "--defined-only", ff.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines()
                if line.split() and line.split()[-2] in ("T", "W")}
    assert exported == set(declared()) == set(ff._SIGNATURES)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_c_consumer(ttc, tmp_path):
    from tiled_tensor_core_05_b200 import ff
    src = tmp_path / "use.c"
    src.write_text('#include <stdio.h>\n#include "gemm_ff.h"\ntypedef void (*fn)(void);\n'
                   "int main(void) {\n  const fn f[] = {" +
                   ", ".join(f"(fn){n}" for n in declared()) + "};\n"
                   '  printf("%d %d %d\\n", (int)(sizeof(f) / sizeof(f[0])), ff_abi_version(),\n'
                   "         ff_gated(0, 0, 0, 0, 0, 0, -1, 1, 8, 8, 8, 8, 8, 8, 8, MX_F16,\n"
                   "                  FF_ACT_SILU, 0));\n  return f[0] == 0;\n}\n")
    exe = tmp_path / "use"
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe), ff.LIB_PATH,
                    f"-Wl,-rpath,{os.path.dirname(ff.LIB_PATH)}"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out == [str(len(declared())), "10000", "-1"]


def test_refusals_before_device_work(ttc):
    lib = ttc.ff_lib()
    n, one = ctypes.c_void_p(0), ctypes.c_void_p(16)
    big = 1 << 31

    def gated(M, F, D, dtype=0, act=3, G=n, U=n):
        return lib.ff_gated(n, n, n, n, G, U, M, F, D, *[8] * 6, dtype, act, None)

    def backward(M, F, D, dtype=0, act=3, dWg=n, dWu=n):
        return lib.ff_gated_backward(*[n] * 9, dWg, dWu, M, F, D, *[8] * 11, dtype, act, None)

    def w4(M, N, K, group=64, dtype=0, act=0):
        return lib.ff_w4_gemm(n, n, n, n, n, n, M, N, K, 8, 16, 8, 16, 8, group, dtype, act, None)

    def w4_gated(M, N, K, group=64, dtype=0, act=0, Zg=n, Zu=n):
        return lib.ff_w4_gated(n, n, n, Zg, n, n, Zu, n, M, N, K, *[16] * 8, group, dtype, act,
                               None)

    for f in (gated, backward, w4, w4_gated):
        for bad in [(-1, 4, 4), (4, -1, 4), (4, 4, -1), (big, 4, 4), (4, big, 4), (4, 4, big),
                    (big - 255, 4, 4)]:
            assert f(*bad) == -1
        for kw in ({"dtype": 2}, {"dtype": -1}, {"act": 4}, {"act": -1}):
            assert f(4, 4, 4, **kw) == -1
    assert gated(4, 4, 4, G=one) == gated(4, 4, 4, U=one) == -1
    assert backward(4, 4, 4, dWg=one) == backward(4, 4, 4, dWu=one) == -1
    for f in (w4, w4_gated):
        for group in (0, 16, 48, 256, -32):
            assert f(4, 4, 4, group=group) == -1
    assert w4_gated(4, 4, 4, Zg=one) == w4_gated(4, 4, 4, Zu=one) == -1
    # nothing to do: whatever the pointers
    assert gated(0, 5, 8) == gated(5, 0, 8) == 0
    assert backward(0, 5, 8) == backward(5, 0, 8) == backward(0, 0, 0) == 0
    assert w4(0, 5, 5) == w4(5, 0, 5) == w4_gated(0, 5, 5) == w4_gated(5, 0, 5) == 0


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (5, 31), (16, 128), (7, 1000)])
def test_layout_of_codes(ttc, rows, cols):
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    for group in (32, 64, 128):
        groups = -(-cols // group)
        codes = torch.randint(0, 16, (rows, cols), generator=g, dtype=torch.uint8)
        scales = torch.rand(rows, groups, generator=g).half()
        zeros = torch.randint(0, 16, (rows, groups), generator=g, dtype=torch.uint8)
        w = ttc.w4_pack(codes, scales, zeros, group=group)
        assert w.shape == (rows, cols) and w.group == group
        words = ref.pack_words(codes.long())
        assert torch.equal(w.data[:, :words.shape[1]], words)
        assert torch.equal(w.scales, scales.t()) and torch.equal(w.zeros, zeros.t())
        assert torch.equal(ttc.w4_unpack(w), codes)
        for t in (w.data, w.scales, w.zeros):
            assert t.shape[0] <= 1 or t.stride(0) * t.element_size() % 16 == 0
        assert ttc.w4_pack(codes, scales, group=group).zeros is None


@pytest.mark.parametrize("rows,cols", [(0, 0), (0, 64), (5, 0)])
def test_layout_of_no_codes(ttc, rows, cols):
    codes = torch.zeros(rows, cols, dtype=torch.uint8)
    zeros = torch.zeros(rows, -(-cols // 32), dtype=torch.uint8)
    w = ttc.w4_pack(codes, zeros.half(), zeros, group=32)
    assert w.shape == (rows, cols) and w.scales.shape == w.zeros.shape == (-(-cols // 32), rows)
    got = ttc.w4_unpack(w)
    assert got.dtype == torch.uint8 and got.shape == (rows, cols)


@pytest.mark.parametrize("rows,groups", [(16, 1), (1, 1), (1, 4), (16, 2), (5, 1)])
def test_packed_weight_is_its_own(ttc, rows, groups):
    """What happens to the codes, scales and zero points afterwards does not reach the weight."""
    codes = torch.full((rows, 32 * groups), 3, dtype=torch.uint8)
    scales, zeros = torch.ones(rows, groups).half(), torch.full((rows, groups), 7).byte()
    w = ttc.w4_pack(codes, scales, zeros, group=32)
    for t in (codes, scales, zeros):
        t.fill_(9)
    assert (ttc.w4_unpack(w) == 3).all() and (w.scales == 1).all() and (w.zeros == 7).all()


def test_word_by_hand():
    """Columns 0 .. 7 of a word: 0, 2, 4, 6 in the low half, 1, 3, 5, 7 in the high half."""
    words = ref.pack_words(torch.arange(8)[None])
    assert words.tolist() == [[0x20, 0x64, 0x31, 0x75]]


def test_python_refusals(ttc):
    codes = torch.zeros(16, 64, dtype=torch.uint8)
    scales = torch.ones(16, 1).half()
    w = ttc.w4_pack(codes, scales, group=64)
    for bad in [(codes.int(), scales), (codes[0], scales)]:
        with pytest.raises(TypeError):
            ttc.w4_pack(*bad, group=64)
    with pytest.raises(TypeError):
        ttc.w4_pack(codes, scales.float(), group=64)
    with pytest.raises(TypeError):
        ttc.w4_pack(codes, scales, torch.zeros(16, 1), group=64)
    for kw in [{"group": 48}, {"group": 32}, {"group": 64, "zeros": torch.zeros(16, 2).byte()},
               {"group": 64, "zeros": torch.full((16, 1), 16).byte()}]:
        with pytest.raises(ValueError):
            ttc.w4_pack(codes, scales, **kw)
    with pytest.raises(ValueError, match="0 .. 15"):
        ttc.w4_pack(codes + 16, scales, group=64)
    args = dict(data=w.data, scales=w.scales, zeros=None, rows=16, cols=64, group=64)
    for key, value in [("rows", 15), ("cols", 65), ("cols", 129), ("group", 16), ("rows", -1),
                       ("scales", w.scales[:, :8]), ("zeros", torch.zeros(1, 15).byte()),
                       ("data", w.data[:, :28]), ("data", torch.zeros(16, 40).byte()),
                       ("data", torch.zeros(32, 16).byte().t()), ("data", w.data[0])]:
        with pytest.raises(ValueError):
            ttc.W4Tensor(**{**args, key: value})
    x = torch.zeros(4, 64).half()
    for f in (lambda: ttc.gemm_w4(x, w), lambda: ttc.gemm_gated_w4(x, w, w),
              lambda: ttc.gemm_gated(x, x, x),
              lambda: ttc.gemm_gated_backward(x, x, x, x, x.float(), x.float())):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    for f in (lambda: ttc.gemm_w4(x, codes), lambda: ttc.gemm_w4(None, w),
              lambda: ttc.gemm_gated_w4(x, w, None), lambda: ttc.gemm_gated(x.float(), x, x),
              lambda: ttc.gemm_gated(None, x, x)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError):
        ttc.gemm_w4(x[:, :32], w)
    other = ttc.w4_pack(codes, scales, torch.zeros(16, 1).byte(), group=64)
    with pytest.raises(ValueError, match="share"):
        ttc.gemm_gated_w4(x, w, other)


# ------------------------------------------------------------- the plain implementation ---


@pytest.mark.parametrize("name", ref.ACTS)
def test_activations_against_torch(name):
    x = torch.linspace(-12, 12, 4801, dtype=torch.float64)
    want = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
            "relu": torch.relu, "none": lambda v: v}[name](x)
    assert (ref.act(x, name) - want).abs().max() < 1e-14
    # the slope against central differences (third derivatives are below 2), off ReLU's corner
    h = 1e-5
    s = (ref.act(x + h, name) - ref.act(x - h, name)) / (2 * h)
    off = (ref.slope(x, name) - s).abs()
    assert off[x.abs() > 2 * h].max() < 1e-9
    assert ref.slope(x, name).abs().max() <= ref.STEEPEST
    bend = (ref.slope(x + h, name) - ref.slope(x - h, name)).abs() / (2 * h)
    assert name == "relu" or bend.max() <= ref.BEND


@pytest.mark.parametrize("name", ref.ACTS)
def test_gradients_against_autograd(name):
    g = torch.Generator().manual_seed(3)
    x, wg, wu = (torch.randn(s, generator=g, dtype=torch.float64, requires_grad=True)
                 for s in ((5, 7), (6, 7), (6, 7)))
    dh = torch.randn(5, 6, generator=g, dtype=torch.float64)
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
         "none": lambda v: v}[name]
    (f(x @ wg.t()) * (x @ wu.t())).backward(dh)
    r = ref.Gated(x.detach(), wg.detach(), wu.detach(), name)
    got = r.backward(dh, torch.float16)
    for k, v in (("dx", x), ("dw_gate", wg), ("dw_up", wu)):
        assert (got[k][0] - v.grad).abs().max() < 1e-13


@pytest.mark.parametrize("group", [32, 64, 128])
def test_weight_by_hand(group):
    codes = torch.arange(300)[None].repeat(2, 1) % 16
    groups = -(-300 // group)
    scales = torch.arange(1.0, 2 * groups + 1).view(groups, 2)
    zeros = torch.arange(2 * groups).view(groups, 2) % 16
    w = ref.weight(codes, scales, zeros, group)
    for n in range(2):
        for k in (0, 31, 32, 64, 127, 128, 299):
            i = k // group
            assert w[n, k] == (k % 16 - (2 * i + n) % 16) * (2 * i + n + 1)
    assert ref.weight(codes, scales, None, group)[1, 5] == (5 - 8) * 2


def test_parts_of_a_weight_cannot_be_exchanged(ttc):
    """A product takes the tensors that were checked: another one in their place is refused."""
    w = ttc.w4_pack(torch.zeros(16, 64, dtype=torch.uint8), torch.ones(16, 1).half(), group=64)
    for name in ("data", "scales", "zeros"):
        with pytest.raises(AttributeError):
            setattr(w, name, getattr(w, name))
    assert w.data.shape == (16, 32) and w.scales.shape == (1, 16) and w.zeros is None


@pytest.mark.parametrize("name", ["rows", "cols", "group"])
def test_sizes_of_a_weight_cannot_be_changed(ttc, name):
    """They were checked together with the tensors, whose extents the library takes from them."""
    w = ttc.w4_pack(torch.zeros(16, 64, dtype=torch.uint8), torch.ones(16, 1).half(), group=64)
    with pytest.raises(AttributeError):
        setattr(w, name, 2 * getattr(w, name))
    assert w.shape == (w.rows, w.cols) == (16, 64) and w.group == 64
