"""Host builds of the fine-tuning library for the CPU checks (test infrastructure).

cases.cpp includes finetune_lib.hip and runs it against the CPU stand-in of
hip/hip_runtime.h in this folder, under AddressSanitizer and
UndefinedBehaviorSanitizer ("asan") or ThreadSanitizer ("tsan").  A build is
redone when any source is newer than its executable.
"""

from __future__ import annotations

import glob
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))
CSRC = os.path.join(ROOT, "block_circulant_layers_amd", "csrc", "finetune")
BUILD = os.path.join(HERE, "_build")
CXX = os.environ.get("RDFFT_HOST_CXX", "/opt/rocm/llvm/bin/clang++")

FLAGS = {
    "tsan": ["-O1", "-g", "-fsanitize=thread"],
    "asan": ["-O1", "-g1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"],
}


def sources():
    return (glob.glob(os.path.join(CSRC, "*.hpp")) + glob.glob(os.path.join(CSRC, "*.hip"))
            + glob.glob(os.path.join(ROOT, "include", "*.h"))
            + [os.path.join(HERE, "cases.cpp"), os.path.join(HERE, "hip", "hip_runtime.h"),
               os.path.join(ROOT, "block_circulant_layers_amd", "csrc", "rdfft_validate.hpp")])


def build(kind: str) -> str:
    exe = os.path.join(BUILD, f"cases_{kind}")
    if os.path.exists(exe) and os.path.getmtime(exe) >= max(os.path.getmtime(s) for s in sources()):
        return exe
    os.makedirs(BUILD, exist_ok=True)
    tmp = exe + ".tmp"
    cmd = [CXX, "-std=c++20", *FLAGS[kind], "-Wno-pass-failed", "-I", HERE, "-I", os.path.join(ROOT, "include"), "-I",
           CSRC, os.path.join(HERE, "cases.cpp"), "-o", tmp, "-lpthread"]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    os.replace(tmp, exe)
    return exe
