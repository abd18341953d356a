"""CPU checks of the fine-tuning kernels' loops over rows and of their forms for
large buffers: the library on CPU threads under the sanitizers, with the numbers
that decide on both made small."""

from __future__ import annotations

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.finetune_check import build_emu


def _build(kind):
    exe = os.path.join(build_emu.BUILD, f"rounds_{kind}")
    src = os.path.join(build_emu.HERE, "rounds.cpp")
    if os.path.exists(exe) and os.path.getmtime(exe) >= max(os.path.getmtime(s) for s in [src, *build_emu.sources()]):
        return exe
    os.makedirs(build_emu.BUILD, exist_ok=True)
    subprocess.run([build_emu.CXX, "-std=c++20", *build_emu.FLAGS[kind], "-O0", "-Wno-pass-failed", "-I", build_emu.HERE, "-I",
                    os.path.join(build_emu.ROOT, "include"), "-I", build_emu.CSRC, src, "-o", exe + ".tmp", "-lpthread"],
                   check=True, capture_output=True, text=True)
    os.replace(exe + ".tmp", exe)
    return exe


def _run(kind):
    return subprocess.run([_build(kind), "small"], capture_output=True, text=True, timeout=900,
                          env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))


@pytest.fixture(scope="module")
def runs():
    with ThreadPoolExecutor() as pool:
        return dict(zip(build_emu.FLAGS, pool.map(_run, build_emu.FLAGS)))


@pytest.mark.parametrize("kind", sorted(build_emu.FLAGS))
def test_rounds_on_cpu_threads(runs, kind):
    r = runs[kind]
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[:4000]
    assert re.match(r"ok 17 \d+\n", r.stdout), r.stdout
