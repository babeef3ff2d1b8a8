"""What build() compiles and links again, and when (CPU; the compilers are stand-ins that touch their output)."""

import os
import subprocess
import time

import pytest
import torch

from sparse_attention_indexer_top_gb300 import build as B


@pytest.fixture()
def commands(tmp_path, monkeypatch):
    """A build folder of its own, and the list of commands that build() has run."""
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libsai.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_binding.so"))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        time.sleep(0.01)  # outputs of later commands are newer
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    return ran


def _links(ran):
    return [c for c in ran if c[0] == "g++" and "-shared" in c]


def _compiles(ran):
    return [c for c in ran if c[-1].endswith(".o") and "binding.cpp" in " ".join(c)]


def test_nothing_is_built_twice(commands):
    B.build()
    assert len(_links(commands)) == 1 and len(_compiles(commands)) == 1
    commands.clear()
    B.build()
    assert commands == []


def test_the_binding_follows_torch_there_and_back(commands, monkeypatch):
    """The module that is there is linked from the object of the torch that imports it."""
    linked = []
    for version in ("9.1", "9.2", "9.1"):
        commands.clear()
        monkeypatch.setattr(torch, "__version__", version)
        B.build()
        with open(B.BINDING) as f:
            linked.append(f"binding-torch-{version}" in f.read())
    assert linked == [True, True, True]
    commands.clear()
    B.build()
    assert commands == []


def test_force_compiles_the_binding_too(commands):
    B.build()
    commands.clear()
    B.build(force=True)
    assert len(_compiles(commands)) == 1 and len(_links(commands)) == 1
