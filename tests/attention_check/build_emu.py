"""Host builds of the sublayer operators for the CPU checks (test infrastructure).

cases.cpp includes attention_lib.hip and the attention kernels and runs them
against the CPU stand-in of hip/hip_runtime.h in this folder, under
AddressSanitizer and UndefinedBehaviorSanitizer ("asan") or ThreadSanitizer
("tsan").  A build is redone when any source is newer than its executable.
"""

from __future__ import annotations

import glob
import os
import subprocess

from tests.finetune_check.build_emu import CSRC, CXX, FLAGS, ROOT

HERE = os.path.dirname(os.path.abspath(__file__))
BUILD = os.path.join(HERE, "_build")


def sources():
    return (glob.glob(os.path.join(CSRC, "*.hpp")) + glob.glob(os.path.join(CSRC, "*.hip"))
            + glob.glob(os.path.join(ROOT, "include", "*.h"))
            + [os.path.join(HERE, "cases.cpp"), os.path.join(HERE, "hip", "hip_runtime.h"),
               os.path.join(ROOT, "tests", "finetune_check", "hip", "hip_runtime.h")])


def build(kind: str) -> str:
    exe = os.path.join(BUILD, f"cases_{kind}")
    if os.path.exists(exe) and os.path.getmtime(exe) >= max(os.path.getmtime(s) for s in sources()):
        return exe
    os.makedirs(BUILD, exist_ok=True)
    tmp = exe + ".tmp"
    cmd = [CXX, "-std=c++20", *FLAGS[kind], "-Wno-pass-failed", "-I", HERE, "-I", os.path.join(ROOT, "include"), "-I",
           CSRC, os.path.join(HERE, "cases.cpp"), "-o", tmp, "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[:6000]
    os.replace(tmp, exe)
    return exe
