"""The suites of the norm, rotation and move of Q, K and V and of the LM-head loss
again, in a child process that loads the bounds-checked debug build: every case
must match as before and no check may fire."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layer_suites_under_the_debug_build(uly):
    if uly.debug_build_selected():
        pytest.skip("already inside the debug-build process")
    from long_context_sequence_head_gb300 import build as b
    b.build(debug=True)
    env = dict(os.environ, ULY_DEBUG_BUILD="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_qkv_norm_rope_gpu.py", "tests/test_linear_ce_gpu.py", "tests/test_linear_ce_label_gpu.py",
           "tests/test_layer_step_gpu.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout, r.stdout[-2000:]
