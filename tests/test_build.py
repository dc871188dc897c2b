"""The library is built with nvcc alone; the native binding of the paged calls where PyTorch's and Python's headers
are installed."""
import subprocess
import sys
import sysconfig

import pytest

import gqa_decode_blackwell_gb300 as g
from gqa_decode_blackwell_gb300 import build as gbuild


@pytest.fixture
def library(monkeypatch):
    """What is asked of nvcc, and what of g++, instead of the building."""
    asked = []
    monkeypatch.setattr(gbuild, "_build_library", lambda *a: asked.append("library") or gbuild.LIB)
    monkeypatch.setattr(gbuild.subprocess, "Popen", lambda *a, **k: pytest.fail("the binding is compiled"))
    return asked


@pytest.mark.parametrize("force", [False, True])
def test_the_library_needs_no_pytorch(library, monkeypatch, force):
    monkeypatch.setitem(sys.modules, "torch", None)                   # import torch raises ImportError
    with pytest.warns(UserWarning, match="paged"):
        assert gbuild.build(force=force) == gbuild.LIB
    assert library == ["library"]


def test_the_library_needs_no_python_headers(library, monkeypatch, tmp_path):
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a: {"include": str(tmp_path)})
    with pytest.warns(UserWarning, match="paged"):
        assert gbuild.build(force=True) == gbuild.LIB
    assert library == ["library"]


def test_a_binding_that_does_not_compile_is_an_error(library, monkeypatch, tmp_path):
    """With all headers there, and whether or not the library was built."""
    monkeypatch.setattr(gbuild, "_start_binding", lambda out, includes: _failed())
    with pytest.raises(subprocess.CalledProcessError):
        gbuild.build(force=True)
    assert library == ["library"]


def _failed():
    class Process:
        returncode = 1

        def wait(self):
            return 1
    return Process()


def test_paged_calls_without_a_binding_say_so(monkeypatch, tmp_path):
    gbuild.build()
    monkeypatch.setattr(g, "_binding", None)
    monkeypatch.setattr(g, "_bound", None)
    monkeypatch.setattr(g, "binding_path", lambda: str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="not built"):
        g._paged()
