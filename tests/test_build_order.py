"""The C library needs hipcc alone: it is linked and put in place whatever becomes of the Python
binding (torch's headers, a host compiler).  The compilers are replaced by a recorder."""
from __future__ import annotations

import os
import sys

import pytest

from parameter_efficient_fine_dora_amd import build


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """build() into tmp_path; returns the commands that ran, and a place for one that fails."""
    ran, broken = [], []

    def run(cmd):
        ran.append(cmd)
        if any(b in arg for b in broken for arg in cmd):
            return 1, "it broke"
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return 0, ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libdora.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / "_bind.so"))
    for name in ("libdora.so", "_bind.so"):
        (tmp_path / name).write_text("old")
    return ran, broken, lambda name: (tmp_path / name).read_text()


def test_both(tools):
    _, _, text = tools
    assert build.build() == build.LIB
    assert text("libdora.so") == text("_bind.so") == "new"


def test_a_binding_that_does_not_compile_leaves_the_library_built(tools):
    _, broken, text = tools
    broken.append("bind.cpp")
    with pytest.raises(RuntimeError, match="bind.cpp"):
        build.build()
    assert text("libdora.so") == "new" and text("_bind.so") == "old"


def test_a_library_that_does_not_compile_leaves_both(tools):
    _, broken, text = tools
    broken.append("gemm.hip")
    with pytest.raises(RuntimeError, match="gemm.hip"):
        build.build()
    assert text("libdora.so") == text("_bind.so") == "old"


def test_without_torch_the_library_alone_is_built(tools, monkeypatch, capsys):
    ran, _, text = tools
    monkeypatch.setitem(sys.modules, "torch", None)     # import torch raises ImportError
    assert build.build() == build.LIB
    assert text("libdora.so") == "new" and text("_bind.so") == "old"
    assert not any("bind.cpp" in arg for cmd in ran for arg in cmd)
    assert "torch" in capsys.readouterr().err
    assert os.path.exists(build.LIB)


def test_a_compiler_that_is_missing_fails_its_own_command():
    rc, out = build._run(["/nowhere/g++", "-o", "x"])
    assert rc != 0 and "/nowhere/g++" in out
