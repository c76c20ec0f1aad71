"""The products with activation, residual and experts on the checked build: every bias, column sum and partly stored chunk
whose address the kernel computes lies in its buffer, for rows of none behind the last expert as well."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_products_pass_on_the_checked_build():
    env = dict(os.environ, BSQ_LIBRARY="checked")
    cmd = [sys.executable, "-m", "pytest", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider", "-k", "not 32_bits",
           os.path.join("tests", "test_gpu_linear.py"), os.path.join("tests", "test_gpu_linear_calls.py")]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert " passed" in r.stdout and "failed" not in r.stdout
