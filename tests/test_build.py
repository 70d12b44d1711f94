"""What the build makes, with compilers that only write down what they are asked for."""

import importlib.util
import os
import types

import pytest

from paged_expert_moe_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of two sources, without results, and a torch of some version."""
    for d in ("pkg/csrc", "include", "torch"):
        (tmp_path / d).mkdir(parents=True)
    for f in ("pkg/csrc/a.cu", "pkg/csrc/b.cu", "pkg/csrc/binding.cpp", "pkg/csrc/x.h", "pkg/csrc/y.cuh", "include/p.h"):
        (tmp_path / f).write_text("")
    (tmp_path / "torch/version.py").write_text("1")
    here = str(tmp_path / "pkg")
    for name, path in (("HERE", here), ("CSRC", here + "/csrc"), ("BUILD", here + "/_build"), ("LIB", here + "/lib.so"),
                       ("BINDING_SRC", here + "/csrc/binding.cpp"), ("BINDING", here + "/_binding.so")):
        monkeypatch.setattr(b, name, path)
    ran = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        ran.append(os.path.basename(out).removesuffix(".tmp"))
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b.subprocess, "run", run)
    t = types.SimpleNamespace(path=tmp_path, ran=ran, torch=str(tmp_path / "torch"))
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name: t.torch and types.SimpleNamespace(submodule_search_locations=[t.torch]))
    return t


def newer(tree, name):
    """The file `name` as if written after everything that was built."""
    t = max(p.stat().st_mtime for p in tree.path.rglob("*")) + 10
    os.utime(tree.path / name, (t, t))


def built(tree, **how):
    del tree.ran[:]
    assert b.build(**how) == b.LIB
    return sorted(tree.ran)


ALL = ["_binding.so", "a.cu.o", "b.cu.o", "lib.so"]


def test_everything_once(tree):
    assert b.needs_build()
    assert built(tree) == ALL
    assert not b.needs_build() and built(tree) == []
    assert built(tree, force=True) == ALL


def test_the_library_needs_no_torch(tree):
    tree.torch = None
    assert b.needs_build()
    assert built(tree) == ALL[1:]
    assert not b.needs_build() and built(tree) == []
    assert built(tree, force=True) == ALL[1:]


def test_torch_that_comes_later_or_changes_rebuilds_the_binding(tree):
    torch, tree.torch = tree.torch, None
    built(tree)
    tree.torch = torch
    assert b.needs_build() and built(tree) == ["_binding.so"]
    (tree.path / "torch/version.py").write_text("2")
    assert b.needs_build() and built(tree) == ["_binding.so"]
    assert not b.needs_build()


@pytest.mark.parametrize("name,what", [("pkg/csrc/a.cu", ALL[1:]), ("pkg/csrc/y.cuh", ALL[1:]), ("pkg/csrc/x.h", ALL),
                                       ("include/p.h", ALL), ("pkg/csrc/binding.cpp", ["_binding.so"])])
def test_a_newer_source_rebuilds_what_is_made_of_it(tree, name, what):
    built(tree)
    newer(tree, name)
    assert b.needs_build() and built(tree) == what
