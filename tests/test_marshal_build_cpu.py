"""The marshalling module is loaded only where it was built for this PyTorch and this
Python, and the library's build does without it."""
import os
import shutil

import pytest
import torch

from allreduce_residual_rmsnorm_gb300 import binding as B
from allreduce_residual_rmsnorm_gb300 import build as BUILD


@pytest.fixture
def built(monkeypatch):
    """The library loaded, the module built and loaded; both as before afterwards."""
    BUILD.build()
    L = B.load()
    if not os.path.exists(BUILD.marshal_path()):
        pytest.skip("marshal.cpp was not built")
    monkeypatch.setattr(B, "_native", None)
    return L


def test_the_module_of_this_version_is_loaded(built):
    B._load_native(built)
    assert B._native is not None


@pytest.mark.parametrize("what", ["version", "commit", "abi", "python"])
def test_a_module_of_another_version_is_not(built, monkeypatch, what):
    here = BUILD.marshal_path()
    if what == "version":
        monkeypatch.setattr(torch, "__version__", "2.99.0")
    elif what == "commit":
        monkeypatch.setattr(torch.version, "git_version", "0" * 40)
    elif what == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI",
                            not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        monkeypatch.setattr(BUILD.sysconfig, "get_config_var", lambda name: "cpython-399")
    assert BUILD.marshal_path() != here
    B._load_native(built)
    assert B._native is None


def test_a_module_without_a_version_in_its_name_is_not(built, monkeypatch, tmp_path):
    shutil.copy(BUILD.marshal_path(), tmp_path / "_marshal.so")
    monkeypatch.setattr(BUILD, "HERE", str(tmp_path))
    B._load_native(built)
    assert B._native is None


def test_build_without_a_host_compiler(monkeypatch, tmp_path, capfd):
    monkeypatch.setattr(BUILD, "HERE", str(tmp_path))
    monkeypatch.setattr(BUILD, "build_library", lambda *a: BUILD.LIB)
    monkeypatch.setattr(BUILD, "marshal_command", lambda out: [str(tmp_path / "no-such-compiler")])
    assert BUILD.build() == BUILD.LIB
    assert "not built" in capfd.readouterr().err
    assert not os.path.exists(BUILD.marshal_path())
    assert BUILD.build() == BUILD.LIB               # not tried again
    assert "not built" not in capfd.readouterr().err


def test_build_without_pytorch(monkeypatch, capfd):
    def no_torch():
        raise ImportError("no torch here")
    monkeypatch.setattr(BUILD, "marshal_path", no_torch)
    monkeypatch.setattr(BUILD, "build_library", lambda *a: BUILD.LIB)
    assert BUILD.build() == BUILD.LIB
    assert "no torch here" in capfd.readouterr().err


def test_an_older_module_does_not_outlive_a_failed_build(monkeypatch, tmp_path):
    monkeypatch.setattr(BUILD, "HERE", str(tmp_path))
    monkeypatch.setattr(BUILD, "build_library", lambda *a: BUILD.LIB)
    monkeypatch.setattr(BUILD, "marshal_command", lambda out: ["false"])
    with open(BUILD.marshal_path(), "wb") as f:
        f.write(b"older")
    os.utime(BUILD.marshal_path(), (0, 0))
    BUILD.build()
    assert not os.path.exists(BUILD.marshal_path())
