"""Large page plans and tables that hold free pages in the bounds-checked build: their own tests once more, in a process of their
own."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_bounds_checked_build():
    files = [os.path.join(TESTS, f) for f in ("test_gpu_pages_large.py", "test_pages_limits.py", "test_gpu_pages_free_entries.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", *files, "-m", "gpu", "-x", "-q", "--bounds-checked", "-p", "no:cacheprovider"],
                       cwd=os.path.dirname(TESTS), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout
