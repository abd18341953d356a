"""The sublayer kernels on CPU threads under the sanitizers: bounds of every
buffer, the LDS schedule, and the borders of the position buckets."""

from __future__ import annotations

import os
import re
import subprocess

import pytest

from tests.attention_check import build_emu


@pytest.mark.parametrize("kind,env", [("asan", {"ASAN_OPTIONS": "detect_leaks=0"}), ("tsan", {})])
def test_kernels_on_cpu_threads(kind, env):
    r = subprocess.run([build_emu.build(kind)], capture_output=True, text=True, timeout=900, env=dict(os.environ, **env))
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[:4000]
    assert re.match(r"ok 16 \d+\n", r.stdout), r.stdout
