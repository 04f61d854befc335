"""Building: the C library needs nvcc alone; the module _fast needs torch and Python's headers, and is left out
without them."""
import os
import subprocess

import pytest

from flashattention_bf16_fwd_b200 import build as fa_build


@pytest.fixture
def ran(monkeypatch):
    commands = []
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: commands.append(cmd))
    return commands


def test_both(ran):
    assert fa_build.build(force=True) == fa_build.LIB
    assert [os.path.basename(c[0]) for c in ran] == ["nvcc", "g++"]


def test_without_torch(ran, monkeypatch, capsys):
    monkeypatch.setitem(__import__("sys").modules, "torch", None)          # import torch raises
    assert fa_build.build(force=True) == fa_build.LIB
    assert [os.path.basename(c[0]) for c in ran] == ["nvcc"]
    assert "torch" in capsys.readouterr().err


def test_without_python_headers(ran, monkeypatch, tmp_path, capsys):
    paths = dict(fa_build.sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(fa_build.sysconfig, "get_paths", lambda: paths)
    assert fa_build.build(force=True) == fa_build.LIB
    assert [os.path.basename(c[0]) for c in ran] == ["nvcc"]
    assert "Python.h" in capsys.readouterr().err


def test_a_failed_compilation_is_raised(monkeypatch):
    def run(cmd, **kw):
        if cmd[0] == "g++":
            raise subprocess.CalledProcessError(1, cmd)
    monkeypatch.setattr(subprocess, "run", run)
    with pytest.raises(subprocess.CalledProcessError):
        fa_build.build(force=True)
