"""build.py without a compiler: what is built when."""
import importlib.metadata
import importlib.util
import os
import subprocess
import types

import pytest

import awq_int4_moe_gb300.build as b


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """Builds into an empty folder; a command makes its output as an empty file."""
    log = []

    def run(cmd, **kw):
        log.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BIND", str(tmp_path / "bind.so"))
    monkeypatch.setattr(subprocess, "run", run)
    return log


def of_binding(log):
    return [c for c in log if any(str(w).endswith("awq_bind.cpp") for w in c)]


def test_library_is_built_where_torch_is_not_installed(commands, monkeypatch, capsys):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not of_binding(commands) and not os.path.exists(b.BIND)
    assert "torch" in capsys.readouterr().err


def test_binding_is_built_again_for_another_torch(commands, monkeypatch):
    b.build()
    assert len(of_binding(commands)) == 1 and os.path.exists(b.BIND)
    b.build()
    assert len(of_binding(commands)) == 1                     # nothing has changed
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.1" if name == "torch" else real(name))
    before = len(commands)
    b.build()
    assert len(of_binding(commands)) == 2
    assert len(commands) == before + 2                        # the binding's compilation and its link, nothing else
