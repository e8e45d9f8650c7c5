"""The build's own bookkeeping: what is compiled again, and when."""
import os
import subprocess
import types

import pytest
import torch

from variable_size_expert_gb300 import build


@pytest.fixture
def compiles(tmp_path, monkeypatch):
    """Compiler commands, not run: the object appears as if they had been."""
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(subprocess, "run", run)
    return ran


def test_python_entry_is_compiled_for_each_torch(compiles, monkeypatch):
    first = build._compile_host()
    assert len(compiles) == 1 and os.path.exists(first)
    assert build._compile_host() == first and len(compiles) == 1       # nothing changed
    here = torch.__version__
    monkeypatch.setattr(torch, "__version__", "99.1.0+other")
    other = build._compile_host()
    assert len(compiles) == 2 and other != first
    monkeypatch.setattr(torch, "__version__", here)
    assert build._compile_host() == first and len(compiles) == 2


def test_python_entry_is_compiled_for_each_source(compiles, monkeypatch):
    obj = build._compile_host()
    os.utime(obj, (1, 1))       # older than host.cpp
    assert build._compile_host() == obj and len(compiles) == 2
