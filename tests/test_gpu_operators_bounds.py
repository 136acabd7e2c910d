"""The tests of the operators' numbers and of their order hold every check of
the bounds-checked library."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_numbers_and_order_hold_every_bounds_check():
    if os.environ.get("QSA_BOUNDS_CHECKED") == "1":
        pytest.skip("this is the checked run")
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
         "tests/test_gpu_dense_numerics.py", "tests/test_gpu_prologue_numerics.py",
         "tests/test_gpu_step_order.py"],
        cwd=ROOT, env=dict(os.environ, QSA_BOUNDS_CHECKED="1"), capture_output=True, text=True,
        timeout=900)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
