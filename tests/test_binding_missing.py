"""The module of csrc/binding.cpp saves time and nothing else: without it the library is built and loaded all the same, and says so."""

import os
import subprocess
import sys

import pytest

from orpo_preference_loss_gb300 import build as orpo_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys, warnings
import torch
import orpo_preference_loss_gb300 as orpo
from orpo_preference_loss_gb300 import build
build.binding_path = lambda debug=False: sys.argv[1]
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    assert orpo.orpo_head_workspace_bytes(64, 1000, 64) > 0
    assert orpo.orpo_pages_workspace_bytes(8, 100, 16, 1) > 0
assert [w for w in seen if issubclass(w.category, RuntimeWarning) and "binding" in str(w.message)], seen
t, one = torch.zeros((2, 64), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
for call in (lambda: orpo.orpo_logits_adjust(t.float(), 2, one, t, one), lambda: orpo.orpo_beam_history(t, t[:1, :2], t[:1, :2], one, one),
             lambda: orpo.orpo_pages_advance(t, one, 16, None, one, None, 1, t[:, :3], one, one, one),
             lambda: orpo.orpo_pages_copy(t.view(1, 2, 1, 16, 4), t[:, :3], one, one), lambda: orpo.orpo_pages_release(t, one, None, one),
             lambda: orpo.orpo_pages_compact(t, one, 16, t, one, one, t[:, :3], one, one, one)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e), e
    else:
        raise AssertionError("host tensors were taken")
print("loaded without")
"""


@pytest.mark.parametrize("content", [None, b"", b"not a module"])
def test_the_library_loads_without(tmp_path, content):
    orpo_build.build()
    path = tmp_path / "orpo_binding-other.so"
    if content is not None:
        path.write_bytes(content)
    r = subprocess.run([sys.executable, "-c", CHILD, str(path)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "loaded without" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("command", [["false"], ["/nowhere/no-such-compiler"]])
@pytest.mark.parametrize("stale", [False, True])
def test_the_library_is_built_without(tmp_path, monkeypatch, command, stale):
    """One of an earlier build goes too: it may not fit the library's entry points any more."""
    lib = orpo_build.build()
    when = os.path.getmtime(lib)
    path = tmp_path / "orpo_binding-other.so"
    if stale:
        path.write_bytes(b"of an earlier build")
        os.utime(path, (0, 0))
    monkeypatch.setattr(orpo_build, "binding_path", lambda debug=False: str(path))
    monkeypatch.setattr(orpo_build, "_binding_command", lambda out: command)
    with pytest.warns(RuntimeWarning, match="binding"):
        assert orpo_build.build() == lib
    assert os.path.getmtime(lib) == when and not path.exists()
