"""Building the library on the CPU: it needs hipcc alone; the CPython module beside it needs torch, and
its failure neither hides nor undoes the library.  (One small source stands for all of them.)"""
import ctypes
import importlib.util
import os
import shutil

import pytest

from moe_grouped_gemm_block_amd import build as b

pytestmark = pytest.mark.skipif(not (os.path.exists(b.HIPCC) or shutil.which(b.HIPCC)), reason="no ROCm toolchain")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    monkeypatch.setattr(b, "SOURCES", ["fp8bs_planner.cpp"])
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib" / "libfp8bs.so"))
    monkeypatch.setattr(b, "MODULE", str(tmp_path / "lib" / "fp8bs_layer_py.so"))
    os.makedirs(b.LIBDIR)
    with open(b.MODULE, "w") as f:
        f.write("an older one")
    return tmp_path


def without_torch(monkeypatch):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))


def test_the_library_needs_no_torch(tree, monkeypatch, capsys):
    without_torch(monkeypatch)
    assert b.build(verbose=True) == b.LIB
    assert os.path.getsize(b.LIB) > 0
    # an older module need not fit the library
    assert not os.path.exists(b.MODULE)
    assert "torch" in capsys.readouterr().out


def test_the_library_is_there_where_the_module_does_not_compile(tree, monkeypatch):
    monkeypatch.setenv("CXX", shutil.which("false"))
    with pytest.raises(RuntimeError, match="fp8bs_layer_py"):
        b.build()
    assert os.path.getsize(b.LIB) > 0 and not os.path.exists(b.MODULE)
    monkeypatch.setenv("CXX", "/nowhere/g++")
    with pytest.raises(RuntimeError, match="fp8bs_layer_py"):
        b.build()
    assert os.path.getsize(b.LIB) > 0


def test_a_module_without_another_compiler(tree, monkeypatch):
    """neither g++ nor c++: hipcc compiles the host code as well"""
    monkeypatch.delenv("CXX", raising=False)
    which, run, used = shutil.which, b.subprocess.run, []
    monkeypatch.setattr(shutil, "which", lambda name, *a: None if name in ("g++", "c++") else which(name, *a))
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: (used.append(cmd[0]), run(cmd, **kw))[1])
    b.build()
    assert set(used) == {b.HIPCC}
    import torch  # noqa: F401  (its libraries)
    assert ctypes.CDLL(b.MODULE).PyInit_fp8bs_layer_py
