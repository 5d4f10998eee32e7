"""What the build makes for whom, without compiling anything."""
import os
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
