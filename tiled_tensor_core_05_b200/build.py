"""Build ``libttc05.so`` (the fp16 GEMM kernels and their C ABI), ``libttcmx.so``
(the microscaled operators) and ``libttcff.so`` (the feed-forward operators)
in-tree with nvcc.

    python -m tiled_tensor_core_05_b200.build [--force] [--verbose] [--ptxas-info]

Every translation unit is compiled for sm_100a only
(``-gencode arch=compute_100a,code=sm_100a``) with ``-lineinfo``, in
parallel, then linked into the shared libraries next to this file.  The CUDA
runtime is linked statically, so the libraries need only the driver at run
time.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libttc05.so")
MX_LIB = os.path.join(PKG, "libttcmx.so")
FF_LIB = os.path.join(PKG, "libttcff.so")
BIND_SOURCES = ["mx_bind.cpp", "ff_bind.cpp"]
COMMON = ["host_common.cu"]  # linked into every library
SOURCES = ["gemm_api.cu", "gemm_tile.cu", "gemm_skinny.cu", "gemm_skinny_even.cu", "gemm_host.cu"]
MX_SOURCES = ["mx_api.cu", "mx_rows.cu", "mx_gemm_split.cu", "mx_gemm_pair.cu",
              "mx_gemm_pair_split.cu"]
FF_SOURCES = ["ff_api.cu", "ff_pair.cu", "ff_split.cu", "ff_rows.cu", "ff_w4.cu",
              "ff_w4_few.cu"]
HEADERS = ["sm100.cuh", "extent.h", "internal.h", "skinny_common.cuh", "tile_common.cuh",
           "mx_internal.h", "mx_common.cuh", "mx_umma.cuh", "ff_internal.h", "ff_common.cuh",
           "bind_common.h"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def bind_path() -> str:
    """The CPython bindings of libttcmx and libttcff, in one file, for the interpreter and the torch
    in use: its name holds what it is compiled against, so that another version builds, and loads,
    one of its own."""
    import sysconfig

    import torch
    return os.path.join(PKG, f"_mxbind.torch{torch.__version__}"
                        f".cxx11abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
                        + sysconfig.get_config_var("EXT_SUFFIX"))


def _inputs():
    files = [os.path.join(CSRC, s)
             for s in COMMON + SOURCES + MX_SOURCES + FF_SOURCES + HEADERS + BIND_SOURCES]
    files += [os.path.join(INCLUDE, h) for h in ("gemm_f16.h", "gemm_mx.h", "gemm_ff.h")]
    files.append(os.path.abspath(__file__))
    return files


def needs_build() -> bool:
    try:
        built = (LIB, MX_LIB, FF_LIB, bind_path())
    except ImportError:  # no torch: the binding has yet to be built
        return True
    if not all(os.path.exists(f) for f in built):
        return True
    t = min(os.path.getmtime(f) for f in built)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _compile(src: str, ptxas_info: bool, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    if ptxas_info:
        cmd += ["-Xptxas", "-v"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if ptxas_info or verbose:
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not ptxas_info and not needs_build():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    sources = COMMON + SOURCES + MX_SOURCES + FF_SOURCES
    with cf.ThreadPoolExecutor(max_workers=len(sources) + 1) as ex:
        bind = ex.submit(_build_bind, verbose)
        objs = dict(zip(sources, ex.map(lambda s: _compile(s, ptxas_info, verbose), sources)))
        ff = ex.submit(_link_library, FF_LIB, [objs[s] for s in COMMON + FF_SOURCES], "ff_*",
                       verbose)
    # only the extern "C" API is exported: gemm_* of libttc05, mx_* of libttcmx, ff_* of libttcff
    _link(MX_LIB, [objs[s] for s in COMMON + MX_SOURCES], "mx_*", verbose)
    _link(LIB, [objs[s] for s in COMMON + SOURCES], "gemm_*", verbose)
    # the binding needs g++ and torch's headers, which the libraries do not; a library's error comes
    # with the binding's, if both failed
    errors = [e for e in (bind.exception(), ff.exception()) if e is not None]
    if errors:
        raise errors[0] from (errors[1] if errors[1:] else None)
    return LIB


def _build_bind(verbose: bool) -> None:
    """The CPython extension: host code only, compiled against the installed torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    lib_dir = cpp_extension.library_paths()[0]
    bind = bind_path()
    tmp = bind + f".tmp{os.getpid()}"
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-I", cuda]
    for d in cpp_extension.include_paths():
        cmd += ["-I", d]
    cmd += [os.path.join(CSRC, f) for f in BIND_SOURCES]
    cmd += ["-o", tmp, "-L", lib_dir, f"-Wl,-rpath,{lib_dir}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BIND_SOURCES}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, bind)


def _link(lib: str, objs: list, exports: str, verbose: bool) -> None:
    _link_library(lib, objs, exports, verbose)


def _link_library(lib: str, objs: list, exports: str, verbose: bool) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    vs = os.path.join(BUILD_DIR, os.path.basename(lib) + ".map")
    with open(vs, "w") as f:
        f.write("{ global: %s; local: *; };\n" % exports)
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + [
        "-Xlinker", f"--version-script={vs}"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true",
                    help="print registers / shared memory / spills per kernel")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    main()
