"""The decode kernels in the bounds-checked build: no computed index leaves its buffer in any of their forms, and outputs
and status words equal the release build's bit for bit.  The checked library runs in a child process, since one process
binds one variant."""

import os
import subprocess
import sys

import numpy as np
import pytest

import orpo_preference_loss_gb300 as orpo
from decode_bounds_cases import CASES, run_case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
import orpo_preference_loss_gb300 as orpo
from orpo_preference_loss_gb300 import build
build.build(debug=True)
orpo.use_bounds_checked_library()
from decode_bounds_cases import CASES, run_case
for i, c in enumerate(CASES):
    np.savez({out!r} + f"/case{{i}}.npz", **run_case(*c))
print("loaded", orpo.lib_path())
"""


def test_decode_kernels_of_the_bounds_checked_build_match_release(tmp_path):
    code = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), out=str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "liborpo_head_debug.so" in r.stdout
    for i, c in enumerate(CASES):
        checked, release = np.load(tmp_path / f"case{i}.npz"), run_case(*c)
        want = orpo.STATUS_BITS["nonfinite"] if "nan" in c[1] else 0
        assert int(checked["status"][0]) == int(release["status"][0]) == want, (c, orpo.orpo_status_string(int(checked["status"][0])))
        for k in release:
            assert np.array_equal(checked[k], release[k], equal_nan=release[k].dtype.kind == "f"), (c, k)
