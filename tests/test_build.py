"""What the build makes for whom, without compiling anything."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import quantized_exact_attention_gb300 as S
from quantized_exact_attention_gb300 import build as B


def test_a_binding_built_for_another_torch_is_not_used(monkeypatch):
    """It reads tensors by torch's layout: after an upgrade it is stale, and not loaded."""
    B.build()
    assert not B._stale()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    monkeypatch.setattr(S, "_paged", None)
    assert B._stale()
    with pytest.raises(RuntimeError, match="not built for this torch"):
        S._paged_binding()


def test_a_binding_built_for_another_python_is_not_used(monkeypatch):
    B.build()
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    here = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: ".cpython-39-none.so" if n == "EXT_SUFFIX" else here(n))
    monkeypatch.setattr(S, "_paged", None)
    assert B._stale()
    with pytest.raises(RuntimeError, match="not built for this torch and Python"):
        S._paged_binding()
    monkeypatch.undo()
    assert os.path.basename(B.binding_path()).endswith(suffix)


def test_the_binding_of_this_torch_and_python_loads():
    B.build()
    assert S._paged_binding().__file__ == B.binding_path()


@pytest.fixture()
def stubbed(monkeypatch, tmp_path):
    """A build into tmp_path whose compilers only leave their output files."""
    def tool(cmd, **_):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name in ("PKG", "BUILD"):
        monkeypatch.setattr(B, name, str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libsage_gb300.so"))
    monkeypatch.setattr(B.subprocess, "run", tool)
    return tmp_path


def test_the_c_library_is_built_without_torch(monkeypatch, stubbed):
    monkeypatch.setitem(sys.modules, "torch", None)        # import torch raises
    assert B.build(force=True) == str(stubbed / "libsage_gb300.so")
    assert os.path.exists(B.LIB) and not B._stale()
    assert not [f for f in os.listdir(stubbed) if "binding" in f]


def test_a_binding_that_does_not_compile_leaves_the_c_library(monkeypatch, stubbed):
    def no_compiler():
        raise RuntimeError("no C++ compiler found")

    monkeypatch.setattr(B, "_compile_binding", no_compiler)
    with pytest.raises(RuntimeError, match="no C.. compiler"):
        B.build(force=True)
    assert os.path.exists(B.LIB) and B._stale()


def test_a_build_makes_both(stubbed):
    B.build(force=True)
    assert os.path.exists(B.LIB) and os.path.exists(B.binding_path()) and not B._stale()
