"""The bounds-checked build (-DHC_BOUNDS_CHECK) on small cases of the operators of include/hc_serve.h,
in a fresh process: each agrees with its oracle and the status word stays clear."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_serve_cases_under_the_bounds_checked_build():
    from hyper_connection_residual_read_gb300 import build
    path = build.build_bounds_checked()
    r = subprocess.run([sys.executable, os.path.join(HERE, "_bounds_serve_cases.py"), path],
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "all cases passed" in r.stdout
