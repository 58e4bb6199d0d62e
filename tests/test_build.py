"""The build without a compiler run: what is built first, what a missing torch stops, and when the
binding's module is out of date.  CPU only; the compilers are stand-ins."""
import importlib.util
import os
import shutil
import sys
import types

import pytest

import gated_token_recurrence_b200 as gtr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(monkeypatch, tmp_path):
    """build.py with its products under tmp_path; .ran lists the compilers that it called."""
    spec = importlib.util.spec_from_file_location("gtr_build", os.path.join(ROOT, "gated_token_recurrence_b200", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.ran, m.gxx_fails = [], False

    def run(cmd, **kw):
        name = os.path.basename(cmd[0])
        m.ran.append(name)
        bad = name == "g++" and m.gxx_fails
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").write(name)
        return types.SimpleNamespace(returncode=int(bad), stdout=b"no")

    monkeypatch.setattr(m.subprocess, "run", run)
    monkeypatch.setattr(m, "sources", lambda: [])
    monkeypatch.setattr(m, "LIB", str(tmp_path / "libgtr.so"))
    monkeypatch.setattr(m, "TORCH_LIB", str(tmp_path / "_gtr_torch.so"))
    monkeypatch.setattr(m, "OBJDIR", str(tmp_path / "obj"), raising=False)
    return m


def test_library_is_built_without_torch(build, monkeypatch, capfd):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert build.build() == build.LIB
    assert open(build.LIB).read() == "nvcc" and not os.path.exists(build.TORCH_LIB)
    assert "torch" in capfd.readouterr().err


@pytest.mark.parametrize("missing", ["g++", "Python.h"])
def test_library_is_built_without_a_compiler_or_headers_for_the_module(build, monkeypatch, tmp_path, capfd, missing):
    which = shutil.which
    if missing == "g++":
        monkeypatch.setattr(shutil, "which", lambda n, *a, **k: None if n == "g++" else which(n, *a, **k))
    else:
        import sysconfig
        monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    open(build.TORCH_LIB, "w").write("old")
    assert build.build(force=True) == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.TORCH_LIB)  # an outdated module is not left to be loaded
    assert missing in capfd.readouterr().err


def test_library_is_there_when_the_module_fails(build):
    build.gxx_fails = True
    with pytest.raises(RuntimeError):
        build.build()
    assert os.path.exists(build.LIB) and build.ran == ["nvcc", "g++"]


def test_module_is_rebuilt_for_another_torch_only(build, monkeypatch):
    import torch
    build.build()
    assert build.ran == ["nvcc", "g++"]
    build.build()
    assert build.ran == ["nvcc", "g++"]  # everything is there
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build()
    assert build.ran == ["nvcc", "g++", "g++"]
    build.build()
    assert build.ran == ["nvcc", "g++", "g++"]


def test_module_built_for_another_torch_is_not_loaded(monkeypatch):
    import torch
    monkeypatch.setattr(gtr, "_native", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(ImportError, match="0.0.1"):
        gtr._marshal()
    monkeypatch.undo()
    assert gtr._marshal() is not None
