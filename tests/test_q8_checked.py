"""The 8-bit operators in the checked build (libcoda_checked.so): their GPU tests on tensor cores run
again in a child process that loads it; each requires a clean status word."""

import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
def test_products_and_backward_in_the_checked_build():
    env = dict(os.environ, CODA_CHECKED_BUILD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_q8_gpu.py"), "-m", "gpu",
                        "-x", "-q", "-k", "test_product or test_bwd or chain or training"], env=env,
                       capture_output=True, text=True, timeout=900, cwd=os.path.dirname(HERE))
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout, out[-4000:]
