"""The extension module of the paged key-value cache calls and the rest of the library: neither needs the other's build."""
import importlib.machinery
import os
import sys

import pytest
import torch

import tensor_allreduce_residual_gb300 as ar
from tensor_allreduce_residual_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _failing(out):
    raise OSError("no compiler")


@pytest.mark.parametrize("command", [lambda out: [sys.executable, "-c", "raise SystemExit(1)"], _failing])
def test_other_calls_are_built_where_the_extension_module_is_not(monkeypatch, tmp_path, command):
    path = tmp_path / "_binding.so"
    path.write_bytes(b"of older sources")
    monkeypatch.setattr(_build, "binding_path", lambda: str(path))
    monkeypatch.setattr(_build, "_binding_stale", lambda: True)
    monkeypatch.setattr(_build, "_binding_command", command)
    with pytest.warns(UserWarning, match="ar_kv_append"):
        assert _build.build() == _build.LIB
    assert not path.exists()
    monkeypatch.setattr(ar, "_calls", None)
    assert ar.lib().ar_workspace_size(2, 1024, ar.AR_BF16) > 0
    with pytest.raises(RuntimeError, match="is missing"):
        ar.ar_attention_join([], [])


@pytest.mark.parametrize("other", ["torch", "python"])
def test_an_extension_module_of_other_versions_is_not_used(monkeypatch, other):
    path = _build.binding_path()
    assert os.path.exists(path) and not _build._binding_stale()
    if other == "torch":
        monkeypatch.setattr(torch, "__version__", "1.0.0")
    else:
        monkeypatch.setattr(importlib.machinery, "EXTENSION_SUFFIXES", [".cpython-30-none.so"])
    assert _build.binding_path() != path and _build._binding_stale()
    monkeypatch.setattr(ar, "_calls", None)
    with pytest.raises(RuntimeError, match="is missing"):
        ar.ar_attention_join([], [])
