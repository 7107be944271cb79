"""Normalisation, rotary positions and attention in the bounds-checked build: their tests
run again in a child process with DPRC_LIBRARY=debug (a failed check is recorded in the
device error word, which the tests' fixture reads).
"""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_block_operators_pass_in_the_bounds_checked_build():
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu",
         "tests/test_gpu_block_operators.py"],
        cwd=ROOT, env=dict(os.environ, DPRC_LIBRARY="debug"), capture_output=True, text=True,
        timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
