"""Bounds-checked debug build (compiled with -DULY_DEBUG) of the windowed
attention, its decode and the norms around a block: their GPU suites run in a
child process on that build, where every raw-pointer access whose place depends
on data or on the schedule is checked, and no check fires."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_window_and_norm_cases_on_the_debug_build():
    from long_context_sequence_head_gb300 import build as b
    b.build(debug=True)
    env = dict(os.environ, ULY_DEBUG_BUILD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu",
                        "tests/test_window_attn_gpu.py", "tests/test_window_sinks_gpu.py", "tests/test_window_decode_gpu.py",
                        "tests/test_residual_norm_gpu.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
