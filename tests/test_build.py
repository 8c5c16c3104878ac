"""CPU tests of the build script: what is built when, with the compilers faked."""

from __future__ import annotations

import os
import subprocess
import types

import pytest

from reference_sliding_window_b200 import build as b


@pytest.fixture()
def faked(tmp_path, monkeypatch):
    """The build in tmp_path with compilers that write their output file and nothing in it."""
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "librswa.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(subprocess, "run", run)
    return ran


def test_the_library_is_linked_whatever_becomes_of_the_binding(faked, monkeypatch):
    def no_torch(force=False):
        raise ImportError("no torch")
    monkeypatch.setattr(b, "build_binding", no_torch)
    with pytest.raises(ImportError, match="no torch"):
        b.build()
    assert os.path.exists(b.LIB)


def test_the_binding_is_rebuilt_for_another_torch_or_python(faked, monkeypatch):
    def binding_builds():
        faked.clear()
        b.build()
        return sum(b.BINDING_SRC in cmd for cmd in faked)

    assert binding_builds() == 1
    assert binding_builds() == 0
    monkeypatch.setattr(b.importlib.metadata, "version", lambda _: "0.0")
    assert binding_builds() == 1
    assert binding_builds() == 0
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda _: "cpython-00")
    assert binding_builds() == 1
    os.utime(b.BINDING, (0, 0))
    assert binding_builds() == 1
