"""CPU checks of the build's steps: what needs torch and a C++ compiler comes
last and keeps nothing else from being built.  The compilers are replaced by a
recorder; nothing is compiled."""

from __future__ import annotations

import os
import sys

import pytest

from block_circulant_layers_amd import build


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """The outputs of the build's commands, in order, each made as an empty file under tmp_path."""
    done = []

    def run(cmd, check=False, **_):
        if cmd[0] == sys.executable:
            return
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        done.append((os.path.basename(cmd[0]), os.path.basename(out)[: -len(".tmp")]))

    monkeypatch.setattr(build.subprocess, "run", run)
    for name in ("LIB", "FINETUNE_LIB", "FINETUNE_HOST", "PROBE_LIB"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    return done


LIBS = ["librdfft.so", "libfinetune.so", "libstreamprobe.so"]


def test_every_library_before_the_module(steps):
    assert build.build(verbose=False) == build.LIB
    assert [out for _, out in steps] == [*LIBS, "_finetune_host.so"]
    assert os.path.exists(build.FINETUNE_HOST)


@pytest.mark.parametrize("missing", ["torch", "compiler"])
def test_without_torch_or_a_compiler(steps, monkeypatch, capsys, missing):
    open(build.FINETUNE_HOST, "w").close()  # a module of an earlier build
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch.utils", None)
    else:
        monkeypatch.setattr(build, "CXX", "no-such-compiler")
    assert build.build(verbose=False) == build.LIB
    assert [out for _, out in steps] == LIBS
    assert not os.path.exists(build.FINETUNE_HOST)
    assert "_finetune_host.so not built" in capsys.readouterr().out
