"""What the build decides before it compiles anything (nothing is compiled
here): the library needs no torch, the Python binding belongs to one torch."""
import os
import sys
import types

import pytest
import torch

from zero_sharded_optimizer_flatten_gb300 import _build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty build tree whose compilers only write their output files."""
    commands = []

    def run(cmd, **how):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libzero.so"))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_train_ops.so"))
    monkeypatch.setattr(_build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(_build.subprocess, "run", run)
    return commands


def test_the_library_builds_without_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)   # import torch raises
    assert not _build.up_to_date()
    assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING)
    assert not any("train_ops" in part for cmd in tree for part in cmd)
    tree.clear()
    assert _build.up_to_date() and _build.build() == _build.LIB and tree == []
    monkeypatch.setitem(sys.modules, "torch", torch)   # with torch the binding is missing
    assert not _build.up_to_date()
