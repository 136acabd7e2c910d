"""The tests of the 8-bit cache, of dense attention over it and of prompt attention hold every check of the
bounds-checked library."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_cache8_and_prompts_hold_every_bounds_check():
    if os.environ.get("QSA_BOUNDS_CHECKED") == "1":
        pytest.skip("this is the checked run")
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_cache8.py",
         "tests/test_gpu_dense8.py", "tests/test_gpu_prompt.py", "tests/test_gpu_prompt_serving.py"],
        cwd=ROOT, env=dict(os.environ, QSA_BOUNDS_CHECKED="1"), capture_output=True, text=True, timeout=900)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
