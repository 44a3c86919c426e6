"""What the build needs: nvcc for the C library, torch and g++ for the Python
binding alone (no GPU; objects that are up to date are not compiled again)."""

import os
import sys

import pytest

from long_context_mean_b200 import build as B


@pytest.fixture
def fresh(tmp_path, monkeypatch):
    """The library and the binding have yet to be linked, from objects that are up to date."""
    B.build()
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libsparseattn.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_serve.so"))
    return tmp_path


def test_the_library_is_linked_without_torch(fresh, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)     # import torch raises ImportError
    with pytest.warns(UserWarning, match="binding.*torch"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_the_library_is_linked_where_the_binding_has_no_compiler(fresh, monkeypatch):
    which = B.shutil.which
    monkeypatch.setattr(B.shutil, "which", lambda name: None if name == "g++" else which(name))
    with pytest.warns(UserWarning, match=r"g\+\+ not found"):
        B.build()
    assert os.path.exists(B.LIB)


def test_a_binding_that_does_not_compile_is_an_error_behind_the_library(fresh, monkeypatch):
    def fails(verbose=False):
        raise RuntimeError("g++ failed for binding.cpp")
    monkeypatch.setattr(B, "build_binding", fails)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        B.build()
    assert os.path.exists(B.LIB)


def test_the_binding_is_built_again_for_another_torch(tmp_path, monkeypatch):
    import importlib.metadata
    from types import SimpleNamespace
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_serve.so"))
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    runs = []

    def compiled(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return SimpleNamespace(returncode=0)
    monkeypatch.setattr(B.subprocess, "run", compiled)
    for version, n in (("1.0", 1), ("1.0", 1), ("1.1", 2), ("1.1", 2)):
        monkeypatch.setattr(importlib.metadata, "version", lambda name, v=version: v)
        B.build_binding()
        assert len(runs) == n


def test_a_binding_for_another_torch_is_refused(monkeypatch):
    import torch

    from long_context_mean_b200 import sa
    B.build()
    monkeypatch.setattr(sa, "_serve", None)
    sa._binding()
    monkeypatch.setattr(sa, "_serve", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="built for torch"):
        sa._binding()


def test_a_binding_that_does_not_say_its_torch_is_refused(monkeypatch):
    """One built before the version was kept in it."""
    from types import SimpleNamespace

    import long_context_mean_b200 as package
    from long_context_mean_b200 import sa
    B.build()
    monkeypatch.setattr(sa, "_serve", None)
    monkeypatch.setattr(package, "_serve", SimpleNamespace(bind=lambda at: None), raising=False)
    with pytest.raises(RuntimeError, match="unknown version"):
        sa._binding()
