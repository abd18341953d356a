"""CPU checks of the fine-tuning library's launch rules: the rules themselves,
compiled for the host, over every size the C ABI admits."""

from __future__ import annotations

import os
import re
import subprocess

from tests.finetune_check import build_emu


def test_launches_stay_below_the_thread_limit(tmp_path):
    exe = str(tmp_path / "launch_rules")
    subprocess.run([build_emu.CXX, "-std=c++20", "-O0", "-I", build_emu.HERE, "-I",
                    os.path.join(build_emu.ROOT, "include"), "-I", build_emu.CSRC,
                    os.path.join(build_emu.HERE, "launch_rules.cpp"), "-o", exe, "-lpthread"],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and re.match(r"ok \d+ \d+\n", r.stdout), (r.returncode, r.stdout, r.stderr)
