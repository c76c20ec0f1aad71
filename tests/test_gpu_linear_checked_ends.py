"""Segments that begin behind row 0 or end inside a step of the depth, on the checked build: every segment, residual, kept
argument and column sum whose address the kernels compute lies in its buffer."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_products_pass_on_the_checked_build():
    env = dict(os.environ, BSQ_LIBRARY="checked")
    cmd = [sys.executable, "-m", "pytest", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider",
           os.path.join("tests", "test_gpu_linear_lead.py"), os.path.join("tests", "test_gpu_linear_wgrad_ends.py")]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert " passed" in r.stdout and "failed" not in r.stdout
