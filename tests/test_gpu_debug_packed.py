"""The packed and paged calls through the index-checking debug build: their
parity suites in a child process, since the library is chosen at import."""
import os
import subprocess
import sys

import pytest

from helpers import has_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEBUG_LIB = os.path.join(ROOT, "exact_io_aware_65_b200", "libfa_debug.so")


@pytest.mark.gpu
@pytest.mark.skipif(not has_gpu(), reason="needs a B200")
def test_packed_and_paged_suites_on_the_debug_build():
    assert os.path.exists(DEBUG_LIB), "build it with python -m exact_io_aware_65_b200.build --debug-bounds"
    tests = [os.path.join(ROOT, "tests", f) for f in ("test_gpu_packed.py", "test_gpu_paged.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", *tests], cwd=ROOT,
                       env=dict(os.environ, FA_LIBRARY=DEBUG_LIB), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "passed" in r.stdout and "skipped" not in r.stdout
