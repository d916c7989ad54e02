"""The C library builds with nvcc alone; the Python module beside it is left out, with a
warning, where it cannot be built."""
import os
import sys

import pytest

from qkv_projection_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build of one small source into an empty folder, with a module of an earlier build."""
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "_host.so").write_bytes(b"of an earlier build")
    for name, value in dict(CSRC=tmp_path, BUILD=tmp_path / "objects", LIB=tmp_path / "lib.so", SOURCES=["one.cu"],
                            HOST_LIB=tmp_path / "_host.so").items():
        monkeypatch.setattr(build, name, value if isinstance(value, list) else str(value))
    return tmp_path


def left_out(tree, capfd, why):
    assert build.build() == str(tree / "lib.so") and os.path.exists(build.LIB)
    assert not os.path.exists(build.HOST_LIB)
    err = capfd.readouterr().err
    assert "without _host.so" in err and why in err


def test_without_torch(tree, capfd, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    left_out(tree, capfd, "torch cannot be imported")


def test_without_a_part_of_torch(tree, capfd, monkeypatch):
    import torch
    monkeypatch.setattr(torch, "__file__", str(tree / "torch" / "__init__.py"))
    left_out(tree, capfd, "ATen.h is missing")


def test_with_a_failing_compiler(tree, capfd, monkeypatch):
    (tree / "broken.cpp").write_text("#error broken\n")
    monkeypatch.setattr(build, "HOST_SOURCE", str(tree / "broken.cpp"))
    left_out(tree, capfd, "broken")


def test_without_a_compiler(tree, capfd, monkeypatch):
    run = build.subprocess.run

    def no_gxx(cmd, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return run(cmd, **kw)
    monkeypatch.setattr(build.subprocess, "run", no_gxx)
    left_out(tree, capfd, "g++ cannot be run")
