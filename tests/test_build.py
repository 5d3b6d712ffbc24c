"""The C-ABI library needs nvcc only: a machine without g++ on the path, torch
or Python's headers, or a binding that does not compile, does not take it
along."""
import os

import pytest

from aware_expert_routing_gb300 import build as b


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build with another place for what it makes, of one small source."""
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libaware_moe.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "SOURCES", ["static_scratch.cu"])
    return tmp_path


def test_nothing_is_lacking_here():
    assert b.binding_lacks() == ""


@pytest.mark.parametrize("what", ["g++", "torch", "Python.h"])
def test_library_without_the_binding(elsewhere, monkeypatch, capfd, what):
    if what == "g++":
        which = b.shutil.which
        monkeypatch.setattr(b.shutil, "which", lambda x, *a, **k: None if x == "g++" else which(x, *a, **k))
    elif what == "torch":
        monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *a: None)
    else:
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(elsewhere)})
    assert b.build() == str(elsewhere / "libaware_moe.so")
    assert os.path.exists(elsewhere / "libaware_moe.so") and not os.path.exists(elsewhere / "_binding.so")
    assert what in capfd.readouterr().err
    assert b.up_to_date()


def test_a_binding_that_does_not_compile_is_an_error_beside_the_library(elsewhere, monkeypatch):
    def fails(obj):
        raise RuntimeError("g++ failed on binding.cpp")
    monkeypatch.setattr(b, "compile_binding", fails)
    with pytest.raises(RuntimeError):
        b.build()
    assert os.path.exists(elsewhere / "libaware_moe.so")
    assert not b.up_to_date()
