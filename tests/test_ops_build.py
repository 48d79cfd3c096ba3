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
