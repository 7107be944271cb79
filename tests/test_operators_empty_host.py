"""Sizes of nothing, without a GPU: a batch without tokens (Poisson sampling draws
one at times) and widths of zero.  What could end the process runs in a child."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _child(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-800:])
    return r.stdout.split()


@pytest.mark.parametrize("dtype", [0, 1])
def test_workspaces_without_tokens(dtype):
    out = _child(
        "from randomized_norm_clipping_gb300 import binding as b\n"
        "f = b.lib().dprc_linear_workspace_bytes\n"
        "for K, N in ((64, 64), (1, 1), (517, 263), (8192, 2048)):\n"
        f"    print(f({dtype}, 0, K, N, 0), f({dtype}, 0, K, N, 1))")
    assert len(out) == 8 and all(0 < int(v) < 1 << 20 for v in out), out


def test_gradient_call_without_tokens_reaches_its_checks():
    # M = 0 with a workspace that is too small: an error code, on any host
    out = _child(
        "from randomized_norm_clipping_gb300 import binding as b\n"
        "P = 0x10000\n"
        "print(b.lib().dprc_linear_grad(P, P, P, P, 1, 0, 64, 64, 0, 0.0, 1, 1, P, P, P, None, P,"
        " 0, None))")
    assert out == ["5"], out
