"""What build() needs, and what it does without (CPU; the compilers are stood in for)."""

import os
import subprocess

import pytest

from moe_decode_weight_gb300 import api, build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Output paths in a folder of their own, and compilers that only write their output file."""
    for name in ("LIB", "BINDING", "TRACE_LIB"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    return calls


def test_build_makes_library_and_binding(tree):
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    if not os.path.exists(build.BINDING):
        pytest.skip("no C compiler or no Python.h here")
    assert sum("binding.c" in a for c in tree for a in c) == 1


@pytest.mark.parametrize("missing", ["headers", "compiler"])
def test_build_without_what_the_binding_needs_still_makes_the_library(tree, missing, monkeypatch):
    if missing == "headers":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    else:
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    with open(build.BINDING, "w") as f:
        f.write("of an earlier build")
    with pytest.warns(UserWarning, match="_binding.so is not built"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_calls_without_the_binding_say_what_is_missing(tmp_path, monkeypatch):
    monkeypatch.setattr(api, "_bound", None)
    monkeypatch.setattr(api, "_PKG", str(tmp_path))
    with pytest.raises(RuntimeError, match="_binding.so is missing"):
        api._binding()
