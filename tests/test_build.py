"""What is built already is used without a compiler, and wherever the tree lies."""
import os
import shutil

from topology_scheduled_gb300 import build


def _gone(*_):
    raise RuntimeError("not installed")


def test_a_built_library_needs_no_compiler(monkeypatch):
    build.build()
    before = os.stat(build.LIB).st_mtime_ns
    monkeypatch.setattr(build, "_nvcc", _gone)
    monkeypatch.setattr(build.subprocess, "run", _gone)
    assert build.build() == build.LIB and os.stat(build.LIB).st_mtime_ns == before


def test_a_built_tree_may_be_moved(monkeypatch, tmp_path):
    here = build._digest()
    shutil.copytree(build.CSRC, tmp_path / "csrc")
    shutil.copytree(build.INCLUDE, tmp_path / "include")
    headers = [str(tmp_path / os.path.basename(os.path.dirname(h)) / os.path.basename(h)) for h in build.HEADERS]
    monkeypatch.setattr(build, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path / "include"))
    monkeypatch.setattr(build, "HEADERS", headers)
    assert build._digest() == here
    with open(tmp_path / "csrc" / "rotary.cu", "a") as f:  # what changes its sources changes the library
        f.write("\n")
    assert build._digest() != here
