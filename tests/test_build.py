"""What build() makes, with the compilers replaced: libnorm.so without PyTorch, and the binding of
the calls on heads for the PyTorch and Python that are installed."""
import os
import shutil
import sys
import types

import pytest
import torch

from normalization_layernorm_rmsnorm_gb300 import _binding as B
from normalization_layernorm_rmsnorm_gb300 import build as nbuild


@pytest.fixture
def ran(monkeypatch, tmp_path):
    """Commands that build() ran, in an empty build folder; each only makes its output, and g++
    fails without the headers."""
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        dirs = [cmd[i + 1] for i, c in enumerate(cmd) if c in ("-I", "-isystem")]
        if cmd[0] == "g++" and "-c" in cmd:
            for h in ("torch/csrc/autograd/python_variable.h", "Python.h"):
                if not any(os.path.exists(os.path.join(d, h)) for d in dirs):
                    return types.SimpleNamespace(returncode=1, stdout="", stderr=f"{h}: no such file")
        open(out, "w").write("made")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(nbuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(nbuild, "LIB", str(tmp_path / "libnorm.so"))
    monkeypatch.setattr(nbuild, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(nbuild, "subprocess", types.SimpleNamespace(run=run))
    return commands


def bindings(commands):
    return [c for c in commands if c[0] == "g++"]


def test_libnorm_needs_no_pytorch(ran, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert nbuild.build() == nbuild.LIB and os.path.exists(nbuild.LIB)
    assert len(ran) == len(nbuild.SOURCES) + 1 and not bindings(ran)
    del ran[:]
    nbuild.build()  # nothing left to do
    assert not ran


def test_libnorm_needs_no_headers_of_pytorch(ran, monkeypatch, tmp_path):
    monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
    assert os.path.exists(nbuild.build()) and not bindings(ran)


def test_libnorm_needs_no_cuda_in_pytorch(ran, monkeypatch, tmp_path):
    # a PyTorch without CUDA has the headers, and no library to link
    home = tmp_path / "torch"
    home.mkdir()
    (home / "include").symlink_to(os.path.join(os.path.dirname(torch.__file__), "include"))
    monkeypatch.setattr(torch, "__file__", str(home / "__init__.py"))
    assert os.path.exists(nbuild.build()) and not bindings(ran)


def test_libnorm_needs_no_gxx(ran, monkeypatch):
    which = shutil.which
    monkeypatch.setattr(nbuild.shutil, "which", lambda c: None if c == "g++" else which(c))
    assert os.path.exists(nbuild.build()) and not bindings(ran)


def test_the_binding_is_built_where_it_can_be_and_only_once(ran):
    nbuild.build()
    assert len(bindings(ran)) == 2 and len(ran) == len(nbuild.SOURCES) + 3
    del ran[:]
    nbuild.build()
    assert not ran


def test_a_failure_of_the_binding_is_raised_after_libnorm_is_made(ran, monkeypatch):
    def fail(*a):
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(nbuild, "_compile_binding", fail)
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        nbuild.build()
    assert os.path.exists(nbuild.LIB)


@pytest.mark.parametrize("change", ["version", "abi", "python"])
def test_the_binding_of_another_pytorch_or_python_is_neither_kept_nor_loaded(ran, monkeypatch, change):
    nbuild.build()
    del ran[:]
    if change == "version":
        monkeypatch.setattr(torch, "__version__", "2.0.0")
    elif change == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        import sysconfig
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
    with pytest.raises(ImportError, match="python -m normalization_layernorm_rmsnorm_gb300.build"):
        B._heads.__wrapped__()
    nbuild.build()
    assert len(bindings(ran)) == 2 and len(ran) == 2
