"""The module of calls.cpp is optional: the library builds without it, and one
that was compiled against another torch or Python is neither kept nor loaded."""

import os
import subprocess

import pytest

import mamba_selective_scan_core_b200 as mm
from mamba_selective_scan_core_b200 import build as mmbuild


def test_the_library_builds_without_it(monkeypatch, capsys):
    mmbuild.build()
    for error in (FileNotFoundError("g++"), subprocess.CalledProcessError(1, "g++"), ImportError("torch")):
        def fails(*args, error=error):
            raise error

        monkeypatch.setattr(mmbuild, "build_calls", fails)
        assert mmbuild.build() == mmbuild.LIB_PATH
        assert "ctypes" in capsys.readouterr().err


def test_one_for_another_torch(monkeypatch, tmp_path):
    """A module of another torch's is compiled anew, and not loaded where that fails."""
    mmbuild.build()
    assert mmbuild.calls_fit() and mm._Torch().calls is not None
    path = tmp_path / "_calls.so"
    with open(mmbuild.CALLS_PATH, "rb") as f:
        path.write_bytes(f.read())
    monkeypatch.setattr(mmbuild, "CALLS_PATH", str(path))
    assert mmbuild.calls_fit()
    monkeypatch.setattr(mmbuild, "calls_for", lambda: "calls.cpp for torch 0.0.1, cpython-312")
    assert not mmbuild.calls_fit()
    assert mm._Torch().calls is None
    commands = []

    def run(cmd, check):
        commands.append(cmd)
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.raises(subprocess.CalledProcessError):
        mmbuild.build_calls()
    assert len(commands) == 1 and not os.path.exists(path)
