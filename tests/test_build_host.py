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


def test_the_binding_is_rebuilt_for_another_torch(tree, monkeypatch):
    """Its age does not tell: an exchanged torch may be older or newer."""
    _build.build()
    assert _build.up_to_date() and _build.binding_problem() is None
    monkeypatch.setattr(_build, "_torch_version", lambda: "9.9.9")
    assert not _build.up_to_date()
    assert "another torch" in _build.binding_problem()
    tree.clear()
    _build.build()
    assert any("train_ops" in part for cmd in tree for part in cmd)
    assert _build.up_to_date() and _build.binding_problem() is None
    os.remove(_build.BINDING)
    assert "not built" in _build.binding_problem()


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    from zero_sharded_optimizer_flatten_gb300 import train_ops as T
    monkeypatch.setattr(T, "_fast", None)
    monkeypatch.setattr(_build, "_torch_version", lambda: "9.9.9")
    with pytest.raises(RuntimeError, match="build"):
        T.zero_expert_sort(torch.zeros(2, 1, dtype=torch.int32), 2)
