"""The compiled Python binding belongs to the torch that it was built with: another one's module is built anew, and not used."""

import importlib.metadata
import subprocess
import types

import pytest
import torch

import causal_gqa_flashattention_attn_gb300 as attn
from causal_gqa_flashattention_attn_gb300 import _build


@pytest.fixture
def built():
    _build.build()


def _other_torch(monkeypatch):
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.8.7" if name == "torch" else real(name))
    monkeypatch.setattr(torch, "__version__", "9.8.7+cu130")


def test_binding_is_rebuilt_for_another_torch(built, monkeypatch):
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        return types.SimpleNamespace(returncode=1, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    _build.build()                        # nothing is stale
    assert not commands
    _other_torch(monkeypatch)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        _build.build()
    assert [c for c in commands if _build.BINDING_SRC in c]
    assert all(_build.BINDING_SRC in c for c in commands)   # the kernels are not compiled again


def test_binding_of_another_torch_is_not_used(built, monkeypatch):
    monkeypatch.setattr(attn, "_native_module", None)
    _other_torch(monkeypatch)
    with pytest.raises(RuntimeError, match="built for torch"):
        attn._native()
    monkeypatch.undo()
    assert attn._native() is not None
