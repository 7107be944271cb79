"""The operators around the norm path in the bounds-checked build.

tests/test_gpu_operators.py runs again in a child process with
DPRC_LIBRARY=debug: every computed index is checked before its access, a failed
check is recorded in the device error word (and the access skipped), and that
file's fixture reads the word after every test.
"""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_operators_pass_in_the_bounds_checked_build():
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "tests/test_gpu_operators.py"],
        cwd=ROOT, env=dict(os.environ, DPRC_LIBRARY="debug"), capture_output=True, text=True,
        timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
