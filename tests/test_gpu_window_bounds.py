"""The bounds-checked build (-DHC_BOUNDS_CHECK) on small cases of the window operators, in a
fresh process: each agrees with its oracle and the status word stays clear (see
test_gpu_bounds.py, which does the same for the read)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_window_cases_under_the_bounds_checked_build():
    from hyper_connection_residual_read_gb300 import build
    path = build.build_bounds_checked()
    r = subprocess.run([sys.executable, os.path.join(HERE, "_bounds_window_cases.py"), path],
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "all cases passed" in r.stdout
