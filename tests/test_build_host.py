"""The build (int4_moe_expert_gb300/_build.py) with stand-ins for the compilers: the C library needs no
PyTorch, the binding is built for the PyTorch and Python at hand, no compiler is left unwaited."""
import os
import sys
import time

import pytest

from int4_moe_expert_gb300 import _build


class Compiler:
    """Stands for subprocess.Popen: writes the command's output file when it is waited for."""
    started, waited, fail = [], [], ""

    def __init__(self, command, **kw):
        self.command, self.returncode = command, None
        Compiler.started.append(self)

    def communicate(self):
        Compiler.waited.append(self)
        self.returncode = int(bool(Compiler.fail) and any(Compiler.fail in c for c in self.command))
        if self.returncode == 0:
            open(self.command[self.command.index("-o") + 1], "w").close()
        return "output", None


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A tree without built files, and the names of what each build compiles and links."""
    Compiler.started, Compiler.waited, Compiler.fail = [], [], ""
    linked = []

    def run(command, check):
        out = command[command.index("-o") + 1]
        linked.append(os.path.basename(out).split(".so")[0])
        open(out, "w").close()
    monkeypatch.setattr(_build, "BUILD", tmp_path / "_build")
    monkeypatch.setattr(_build, "LIB", tmp_path / "libmoe_gb300.so")
    monkeypatch.setattr(_build, "BINDING", tmp_path / "_moe_torch.so")
    monkeypatch.setattr(_build.subprocess, "Popen", Compiler)
    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "nvcc", lambda: sys.executable)

    def build(**kw):
        Compiler.started, Compiler.waited, linked[:] = [], [], []
        time.sleep(0.01)                       # later files have later times
        _build.build_library(**kw)
        assert Compiler.waited == Compiler.started
        return sorted(os.path.basename(c.command[c.command.index("-c") + 1]) for c in Compiler.started), sorted(linked)
    return build


def test_everything_is_built_once(tree):
    pytest.importorskip("torch")
    if _build.binding_key() is None:
        pytest.skip("PyTorch without CUDA")
    assert tree() == (sorted(_build.SOURCES + ["moe_torch.cpp"]), ["_moe_torch", "libmoe_gb300"])
    assert _build.binding_built_for() == _build.binding_key()
    assert tree() == ([], [])


def test_the_c_library_is_built_without_pytorch(tree, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)        # importing it raises ImportError
    assert _build.binding_key() is None
    assert tree() == (sorted(_build.SOURCES), ["libmoe_gb300"])
    assert "PyTorch" in capsys.readouterr().out and _build.binding_built_for() is None


def test_the_binding_is_built_again_for_another_pytorch_or_python(tree, monkeypatch):
    torch = pytest.importorskip("torch")
    if _build.binding_key() is None:
        pytest.skip("PyTorch without CUDA")
    tree()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert _build.binding_built_for() != _build.binding_key()
    assert tree() == (["moe_torch.cpp"], ["_moe_torch"])
    assert tree() == ([], [])
    import sysconfig
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-999")
    assert tree() == (["moe_torch.cpp"], ["_moe_torch"])


def test_every_compiler_is_waited_for_when_something_fails(tree, monkeypatch):
    Compiler.fail = "moe_fp8.cu"
    with pytest.raises(RuntimeError, match="compilation failed"):
        tree()
    assert len(Compiler.waited) == len(Compiler.started) >= len(_build.SOURCES)

    def broken():
        raise OSError("no such library")
    monkeypatch.setattr(_build, "binding_key", broken)     # after the compilers were started
    with pytest.raises(OSError):
        tree(force=True)
    assert len(Compiler.waited) == len(Compiler.started) == len(_build.SOURCES)
