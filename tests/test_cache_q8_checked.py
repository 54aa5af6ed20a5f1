"""The 8-bit paged cache in the checked build (libcoda_checked.so): its GPU tests run again in a child process that loads
it; each that expects nothing wrong requires a clean status word."""

import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
@pytest.mark.parametrize("file,which", [
    ("test_cache_q8_gpu.py", "test_write or axes or extreme or codes or bad_pages"),
    ("test_attn_q8_gpu.py", "test_attention or bad_pages or before_the_first or 2_31 or layer"),
    ("test_attn_q8_range_gpu.py", "many_batches or unseen"),
    ("test_cache_q8_calls_gpu.py", "nonsense or many_sequences or hints or nothing"),
])
def test_cache_in_the_checked_build(file, which):
    env = dict(os.environ, CODA_CHECKED_BUILD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, file), "-m", "gpu", "-x", "-q", "-k", which],
                       env=env, capture_output=True, text=True, timeout=900, cwd=os.path.dirname(HERE))
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout, out[-4000:]
