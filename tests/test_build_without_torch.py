"""The library is built where the marshalling module cannot be, and the binding does without it (no GPU needed)."""
import importlib.util
import os
import shutil
import sys

import pytest

from differential_attention_04_b200 import _lib
from differential_attention_04_b200 import build as b


@pytest.fixture
def module_at(monkeypatch, tmp_path):
    """A place of its own for the module, with one of older sources in it."""
    b.build()
    at = tmp_path / "_marshal.so"
    at.write_bytes(b"old")
    os.utime(at, (1, 1))
    monkeypatch.setattr(b, "MARSHAL", str(at))
    return at


def _no_torch(m, tmp):
    real = importlib.util.find_spec
    m.setattr(b.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else real(n, *a))


def _no_headers(m, tmp):
    m.setattr(b.sysconfig, "get_paths", lambda *a: {"include": str(tmp)})


def _no_compiler(m, tmp):
    real = shutil.which
    m.setattr(b.shutil, "which", lambda n, *a: None if n == "g++" else real(n, *a))


def _failing_compiler(m, tmp):
    real = shutil.which
    m.setattr(b.shutil, "which", lambda n, *a: real("false" if n == "g++" else n, *a))


@pytest.mark.parametrize("without,says", [(_no_torch, "torch"), (_no_headers, "Python's headers"), (_no_compiler, "g++"),
                                          (_failing_compiler, "g++ failed")])
def test_library_is_built_without_the_module(without, says, module_at, monkeypatch, tmp_path, capfd):
    without(monkeypatch, tmp_path)
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not module_at.exists()  # (it would have been bound to entry points of another header)
    err = capfd.readouterr().err
    assert "marshalling module was not built" in err and says in err
    assert b.build_marshal() is None


def test_binding_does_without_the_module(monkeypatch):
    b.build()
    handle = _lib.lib()
    monkeypatch.setattr(_lib, "_marshal", _lib._marshal)
    monkeypatch.setitem(sys.modules, "differential_attention_04_b200._marshal", None)
    monkeypatch.delattr(sys.modules["differential_attention_04_b200"], "_marshal", raising=False)
    _lib._bind_marshal(handle)
    assert _lib.marshal() is False
