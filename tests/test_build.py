"""The build's optional part, the C++ marshalling module: what it is named, when it is built again,
and that a machine which cannot build it is left with a working library.  Nothing is compiled."""
import os
import subprocess
import sysconfig
import types
import warnings

import pytest

from post_weight_pruning_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package folder, an object folder and a PyTorch of the test's own; `runs` holds the commands."""
    t = types.SimpleNamespace(here=tmp_path / "pkg", runs=[], status=0, error=None)
    for d in ("pkg/csrc", "obj", "torch", "include"):
        (tmp_path / d).mkdir(parents=True)
    (t.here / "csrc" / "fastcall.cpp").write_text("")
    (tmp_path / "include" / "pwp.h").write_text("")
    t.version = tmp_path / "torch" / "version.py"
    t.version.write_text("__version__ = '1'")
    t.module = t.here / os.path.basename(B.FASTCALL)
    for name, path in (("HERE", t.here), ("ROOT", tmp_path), ("CSRC", t.here / "csrc"), ("OBJ", tmp_path / "obj"),
                       ("FASTCALL", t.module)):
        monkeypatch.setattr(B, name, str(path))
    spec = types.SimpleNamespace(origin=str(tmp_path / "torch" / "__init__.py"))
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: spec)
    monkeypatch.setattr(B, "_nvcc", lambda: "/cuda/bin/nvcc")

    def run(cmd, **kw):
        t.runs.append(cmd)
        if t.error is not None:
            raise t.error
        if t.status == 0:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, t.status, "", "cannot find -ltorch_cuda")
    monkeypatch.setattr(B.subprocess, "run", run)
    return t


def test_the_module_is_named_for_its_interpreter():
    assert B.FASTCALL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and "cpython" in os.path.basename(B.FASTCALL)


def test_built_again_for_another_pytorch_or_source(tree):
    build = lambda: B._build_fastcall(False)
    build()
    assert len(tree.runs) == 1 and tree.module.exists()
    build()
    assert len(tree.runs) == 1
    tree.version.write_text("__version__ = '2'")
    build()
    assert len(tree.runs) == 2
    build()
    assert len(tree.runs) == 2
    later = os.path.getmtime(tree.module) + 5
    os.utime(tree.here / "csrc" / "fastcall.cpp", (later, later))
    build()
    assert len(tree.runs) == 3


@pytest.mark.parametrize("error", [None, FileNotFoundError("g++")])
def test_a_machine_that_cannot_build_it_is_warned(tree, error):
    B._build_fastcall(False)
    tree.version.write_text("__version__ = '2'")
    tree.status, tree.error = 1, error
    with pytest.warns(UserWarning, match="not built"):
        B._build_fastcall(False)
    assert not tree.module.exists()                   # the one for the other PyTorch is not left behind
    tree.status, tree.error = 0, None
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        B._build_fastcall(False)
    assert tree.module.exists()


def test_a_module_without_the_tag_is_taken_away(tree):
    old = tree.here / "_fastcall.so"
    old.write_text("")
    B._build_fastcall(False)
    assert not old.exists() and tree.module.exists()


def test_without_pytorch_nothing_is_built(tree, monkeypatch):
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: None)
    B._build_fastcall(False)
    assert not tree.runs
