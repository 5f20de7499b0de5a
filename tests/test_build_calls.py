"""libtsa.so is built and loaded without what tsa_calls.so needs: PyTorch's and Python's headers, and g++ by its name."""
import os
import subprocess

import pytest

import topology_scheduled_gb300 as tsa
from topology_scheduled_gb300 import binding, build


def test_the_library_without_the_calls(monkeypatch, tmp_path):
    tsa.lib()
    ran = []

    def run(cmd, **kw):
        if cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")
        ran.append(os.path.basename(cmd[cmd.index("-o") + 1]))
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name, file in (("LIB", "libtsa.so"), ("CALLS", "tsa_calls.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "_nvcc", lambda: "/opt/cuda/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="calls.cpp"):  # the calls' lack is reported ..
        build.build()
    assert len(ran) == len(build.SOURCES) + 1 and os.path.exists(build.LIB)  # .. with the library there
    ran.clear()
    assert build.build_library() == build.LIB and not ran


def test_loading_the_library_does_not_build_the_calls(monkeypatch):
    def gone(*_, **__):
        raise RuntimeError("not installed")

    tsa.lib()
    monkeypatch.setattr(build, "build_calls", gone)
    monkeypatch.setattr(binding, "_LIB", None)
    monkeypatch.setattr(binding, "_CALLS", None)
    assert tsa.lib().tsa_status_string(0)
    with pytest.raises(RuntimeError, match="not installed"):
        binding.calls()
