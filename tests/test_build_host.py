"""Host tests of the build where the compiled half of the binding cannot be made:
the library is built all the same."""

import importlib.machinery
import os
import subprocess
import sys

import pytest

from tile_size_decision_gb300 import build


@pytest.fixture()
def elsewhere(tmp_path, monkeypatch):
    """The compiled calls and the linked library go to a folder of the test's own."""
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libtiles.so"))
    return tmp_path


def torch_at(monkeypatch, folder):
    spec = importlib.machinery.ModuleSpec("torch", None, origin=str(folder / "__init__.py"))
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda name, *a: spec if name == "torch" else find(name, *a))


def test_a_pytorch_without_cuda(elsewhere, monkeypatch):
    lib = elsewhere / "torch" / "lib"
    lib.mkdir(parents=True)
    (lib / "libtorch_cpu.so").write_bytes(b"")
    (elsewhere / "torch" / "version.py").write_text("")
    torch_at(monkeypatch, elsewhere / "torch")
    (elsewhere / "_calls.so").write_bytes(b"of a PyTorch that was here before")
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)


def test_no_pytorch(elsewhere, monkeypatch):
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)


def test_a_compiler_that_fails_on_the_calls(elsewhere, monkeypatch):
    pytest.importorskip("torch")
    run = subprocess.run

    def failing(cmd, *a, **kw):
        if build.CALLS + ".tmp" in cmd:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        return run(cmd, *a, **kw)

    monkeypatch.setattr(build.subprocess, "run", failing)
    (elsewhere / "_calls.so").write_bytes(b"of other sources")
    os.utime(elsewhere / "_calls.so", (0, 0))
    with pytest.warns(UserWarning, match="no such header"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)


def test_compiled_calls_that_do_not_load(monkeypatch):
    pytest.importorskip("torch")
    import tile_size_decision_gb300 as T
    build.build()
    monkeypatch.setattr(T, "_CALLS", None)
    # What the import system does for a library of another PyTorch.
    monkeypatch.delattr(T, "_calls", raising=False)
    monkeypatch.setitem(sys.modules, T.__name__ + "._calls", None)
    with pytest.warns(UserWarning, match="do not load"):
        assert T._compiled() is T._NoCalls
    assert T._CALLS is T._NoCalls
