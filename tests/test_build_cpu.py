"""The build without a GPU: the C library's users need neither torch nor a compiler of
their own beside hipcc."""
import importlib.util
import os
import subprocess

from linear_layer_amd import _build


def test_no_python_module_without_torch(monkeypatch):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    monkeypatch.setattr(subprocess, "run", lambda *a, **k: (_ for _ in ()).throw(AssertionError("a compiler was called")))
    assert _build._build_call() is False


def test_python_module_takes_hipcc(monkeypatch, tmp_path):
    called = []

    def run(cmd, **k):
        called.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(_build, "CALL", os.path.join(tmp_path, "_call.so"))
    monkeypatch.setenv("CXX", "/nowhere/c++")
    assert _build._build_call() is True
    assert [c[0] for c in called] == [_build.HIPCC] and os.path.exists(_build.CALL)
