"""What build() makes when torch is missing or changes, with the compilers replaced by a stand-in
that writes their outputs."""
import importlib.util
import os
import subprocess
import types

import pytest

from quantized_matmul_gb300 import build


@pytest.fixture
def made(tmp_path, monkeypatch):
    """build's outputs in a folder of their own, and the commands it ran (binding.cpp "fails" if asked)."""
    commands, fail = [], []
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libqmm.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_qmm_torch.so"))
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")

    def run(cmd, **kw):
        commands.append(cmd)
        if fail and any(c.endswith("binding.cpp") for c in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    return types.SimpleNamespace(commands=commands, fail=fail)


def torch_at(monkeypatch, root):
    """The import system finds torch at `root`, or not at all."""
    find = importlib.util.find_spec

    def find_spec(name, *a):
        if name != "torch":
            return find(name, *a)
        return None if root is None else types.SimpleNamespace(origin=str(root / "__init__.py"))

    monkeypatch.setattr(importlib.util, "find_spec", find_spec)


@pytest.fixture
def fake_torch(tmp_path, monkeypatch):
    root = tmp_path / "site" / "torch"
    (root / "include" / "ATen").mkdir(parents=True)
    (root / "include" / "ATen" / "ATen.h").write_text("")
    (root / "version.py").write_text("__version__ = '2.9.1'\n")
    torch_at(monkeypatch, root)
    python = tmp_path / "python"
    python.mkdir()
    (python / "Python.h").write_text("")
    import sysconfig
    monkeypatch.setattr(sysconfig, "get_path", lambda name: str(python))
    return root


def test_without_torch_the_library_is_built_alone(made, monkeypatch, capsys):
    torch_at(monkeypatch, None)
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    err = capsys.readouterr().err
    assert "torch is not installed" in err and "_qmm_torch.so is not built" in err
    assert not build.up_to_date()


def test_without_python_headers_the_library_is_built_alone(made, fake_torch, tmp_path, capsys):
    (tmp_path / "python" / "Python.h").unlink()
    build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "Python.h is missing" in capsys.readouterr().err


def test_a_binding_that_does_not_compile_is_an_error_after_the_library(made, fake_torch):
    made.fail.append(True)
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_a_changed_torch_rebuilds_the_binding_alone(made, fake_torch):
    build.build()
    assert build.up_to_date()
    made.commands.clear()
    build.build()
    assert not made.commands
    (fake_torch / "version.py").write_text("__version__ = '2.11.0'\n")
    assert not build.up_to_date()
    build.build()
    assert [os.path.basename(c[0]) for c in made.commands] == ["g++", "g++"]
    assert build.up_to_date()


def test_a_changed_binding_source_leaves_the_library(made, fake_torch, monkeypatch):
    build.build()
    made.commands.clear()
    later = os.path.getmtime(build.BINDING) + 10
    getmtime = os.path.getmtime
    monkeypatch.setattr(os.path, "getmtime", lambda f: later if str(f).endswith("binding.cpp") else getmtime(f))
    assert build.library_up_to_date() and not build.binding_up_to_date()
    build.build()
    assert [os.path.basename(c[0]) for c in made.commands] == ["g++", "g++"]
