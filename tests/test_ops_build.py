"""The optional torch_calls module: how it is named, built and loaded, and that everything works without it."""
import os
import sysconfig

import pytest

from quantized_moe_decode_softmax_gb300 import build as qbuild
from quantized_moe_decode_softmax_gb300 import ops


def test_module_is_named_for_its_interpreter():
    """Two interpreters with the same torch do not take each other's module."""
    assert qbuild.calls_path().endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.basename(qbuild.calls_path()) != "_torch_calls" + sysconfig.get_config_var("EXT_SUFFIX")


def test_a_module_that_does_not_load_leaves_ctypes(monkeypatch, tmp_path):
    qbuild.build()
    ops._lib()
    bad = tmp_path / "_torch_calls.so"
    bad.write_bytes(b"no shared library")
    monkeypatch.setattr(ops, "_calls", None)
    monkeypatch.setattr(ops, "_c", None)
    monkeypatch.setattr(qbuild, "calls_path", lambda: str(bad))
    with pytest.warns(UserWarning, match="ctypes"):
        assert ops._bind() is ops._c
    assert ops._calls is None


def no_nvcc():
    raise RuntimeError("nvcc not found")


@pytest.mark.parametrize("compiler", ["/nonexistent/c++", "false"])
def test_library_is_built_without_a_host_build_against_torch(monkeypatch, tmp_path, compiler):
    """A missing or failing C++ compiler costs the module alone; a module of older sources
    is taken away, since it may not fit the library any more."""
    qbuild.build()
    path = tmp_path / "_torch_calls.so"
    monkeypatch.setattr(qbuild, "calls_path", lambda: str(path))
    monkeypatch.setenv("CXX", compiler)
    with pytest.warns(UserWarning, match="ctypes"):
        assert qbuild.build() == qbuild.LIB_PATH
    path.write_bytes(b"old")
    os.utime(path, (1, 1))
    with pytest.warns(UserWarning, match="ctypes"):
        assert qbuild.build_calls() is None
    assert not path.exists()


def test_module_needs_no_nvcc(monkeypatch, tmp_path):
    """Another torch beside an up-to-date library asks for the host compiler only."""
    qbuild.build()
    monkeypatch.setattr(qbuild, "calls_path", lambda: str(tmp_path / "_torch_calls.so"))
    monkeypatch.setattr(qbuild, "_nvcc", no_nvcc)
    assert qbuild.build() == qbuild.LIB_PATH and (tmp_path / "_torch_calls.so").exists()
