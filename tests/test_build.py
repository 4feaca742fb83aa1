"""The build of the libraries and of the binding, without compiling anything."""
import os

import pytest

from tiled_tensor_core_05_b200 import build


def test_libraries_do_not_wait_for_the_binding(tmp_path, monkeypatch):
    """Without g++ or torch's headers there is no binding; both libraries, which need nvcc alone,
    are linked all the same, and the binding's error is raised after that."""
    linked = []

    def no_compiler(verbose):
        raise RuntimeError("no g++")

    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "_compile", lambda src, info, verbose: src + ".o")
    monkeypatch.setattr(build, "_link", lambda lib, objs, exports, verbose: linked.append(
        (os.path.basename(lib), exports, sorted(objs))))
    monkeypatch.setattr(build, "_build_bind", no_compiler)
    with pytest.raises(RuntimeError, match="no g"):
        build.build(force=True)
    assert sorted(linked) == [
        ("libttc05.so", "gemm_*", sorted(s + ".o" for s in build.COMMON + build.SOURCES)),
        ("libttcmx.so", "mx_*", sorted(s + ".o" for s in build.COMMON + build.MX_SOURCES))]
