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


def test_binding_of_another_torch_is_not_taken_for_current(tmp_path, monkeypatch):
    """The binding is compiled against one torch and one interpreter: with another version in use
    it is built again, and the old one is not loaded."""
    import torch

    import tiled_tensor_core_05_b200 as ttc
    from tiled_tensor_core_05_b200 import mx
    build.build()
    ttc.mx_lib()
    assert not build.needs_build()
    before = build.bind_path()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.99.0+other")
        assert build.bind_path() != before and build.needs_build()
        m.setattr(mx, "_lib", None)
        m.setattr(mx, "_bind", None)
        with pytest.raises(RuntimeError, match="missing"):
            ttc.mx_lib()
    with monkeypatch.context() as m:
        m.setattr("sysconfig.get_config_var", lambda name: ".cpython-399.so")
        assert build.bind_path() != before and build.needs_build()
    assert not build.needs_build()


def test_build_without_torch_is_not_current(monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert build.needs_build()
