"""What build() asks for, with a compiler that writes empty files: the library needs nvcc alone, its Python binding
PyTorch with CUDA and a C++ compiler beside it."""
import os
import subprocess
import sys
import types

import pytest

from bit_block_scaled_gb300 import build as B


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    """Commands that were run; `fails` names a source or output whose command fails."""
    c = types.SimpleNamespace(ran=[], fails=None)
    for name, path in (("BUILD", "_build"), ("LIB", "libmoe4.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(B, name, str(tmp_path / path))
    monkeypatch.setattr(B, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")

    def run(cmd, **_):
        c.ran.append(cmd)
        bad = c.fails is not None and any(a.endswith(c.fails) for a in cmd)
        if not bad:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write(str(len(c.ran)))
        return subprocess.CompletedProcess(cmd, int(bad), "", "error" if bad else "")
    monkeypatch.setattr(B.subprocess, "run", run)
    return c


def sources(c):
    return sorted(os.path.basename(a) for cmd in c.ran for a in cmd if a.endswith((".cu", ".cpp")))


def test_everything_once(compiler):
    pytest.importorskip("torch")
    B.build()
    assert sources(compiler) == sorted(B.SOURCES + ["binding.cpp"])
    assert os.path.exists(B.LIB) and os.path.exists(B.BINDING)
    compiler.ran.clear()
    B.build()
    assert compiler.ran == []


def no_torch(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)


def torch_without_cuda(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.version, "cuda", None)


def no_compiler(monkeypatch):
    which = B.shutil.which
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(B.shutil, "which", lambda name, *a: None if name == "g++" else which(name, *a))


@pytest.mark.parametrize("without", [no_torch, torch_without_cuda, no_compiler])
def test_the_library_without_what_its_binding_needs(compiler, monkeypatch, without):
    without(monkeypatch)
    assert B.build() == B.LIB
    assert sources(compiler) == sorted(B.SOURCES) and os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    compiler.ran.clear()
    B.build()
    assert compiler.ran == []


def test_a_binding_that_fails_leaves_the_library(compiler):
    pytest.importorskip("torch")
    compiler.fails = "binding.cpp"
    with pytest.raises(RuntimeError):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    compiler.fails = "norm.cu"
    os.remove(os.path.join(B.BUILD, "norm.o"))
    os.remove(B.LIB)
    with pytest.raises(RuntimeError):
        B.build()
    assert not os.path.exists(B.LIB)


@pytest.mark.parametrize("what", ["__version__", "git_version"])
def test_another_torch_rebuilds_the_binding(compiler, monkeypatch, what):
    """Its ABI is that of the PyTorch it was compiled against; the library has nothing to do with it."""
    torch = pytest.importorskip("torch")
    B.build()
    compiler.ran.clear()
    monkeypatch.setattr(*((torch, "__version__") if what == "__version__" else (torch.version, "git_version")), "another")
    B.build()
    assert sources(compiler) == ["binding.cpp"] and len(compiler.ran) == 2
    compiler.ran.clear()
    B.build()
    assert compiler.ran == []


def test_a_binding_that_failed_is_tried_again(compiler):
    pytest.importorskip("torch")
    compiler.fails = B.BINDING + ".tmp"
    with pytest.raises(RuntimeError):
        B.build()
    compiler.fails = None
    B.build()
    assert os.path.exists(B.BINDING)
