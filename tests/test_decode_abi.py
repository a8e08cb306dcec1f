"""Host-side checks of the decode entry points: every refusal returns its code before any CUDA call."""

import ctypes
import math

import pytest
import torch

import orpo_preference_loss_gb300 as orpo
from orpo_preference_loss_gb300 import build as orpo_build

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ARG, ERR_WS = 0, 1, 2, 3, 4, 5
P = lambda a: ctypes.c_void_p(a)  # noqa: E731
FAKE = P(0x10000)  # never dereferenced
MAX_ROWS = (1 << 31) - (1 << 16)


@pytest.fixture(scope="module")
def lib():
    orpo_build.build()
    return orpo.load()


def test_logits_host_checks(lib):
    def call(h=FAKE, ld_h=64, wq=FAKE, sc=FAKE, bi=FAKE, bits=4, group=32, M=2, V=128, d=64, cap=0.0, out=FAKE,
             ld=128, bf16=0, ws=None, ws_bytes=0, st=FAKE):
        return lib.orpo_head_logits_q(h, ld_h, wq, sc, bi, bits, group, M, V, d, cap, out, ld, bf16, ws, ws_bytes, st,
                                      None)

    assert call(M=0) == OK
    for bad in (dict(M=-1), dict(M=MAX_ROWS + 1), dict(V=0), dict(V=MAX_ROWS + 1), dict(d=0), dict(d=1 << 20),
                dict(ld_h=56), dict(ld=127)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in ("h", "wq", "sc", "bi", "out", "st"):
        assert call(**{bad: None}) == ERR_NULL, bad
    for bad in (dict(bits=5), dict(group=12), dict(group=0), dict(group=48), dict(cap=math.nan), dict(cap=math.inf)):
        assert call(**bad) == ERR_ARG, bad
    for bad in (dict(ld_h=68), dict(h=P(0x10008)), dict(wq=P(0x10002)), dict(bits=8, wq=P(0x10004)),
                dict(out=P(0x10002)), dict(out=P(0x10001), bf16=1), dict(sc=P(0x10001))):
        assert call(**bad) == ERR_ALIGN, bad
    # more rows than fit on chip need a workspace
    big = dict(M=17, d=4096, ld_h=4096)
    need = lib.orpo_head_logits_q_workspace_bytes(17, 4096, 4)
    assert need >= 17 * 4096 * 2
    assert call(**big) == ERR_NULL
    assert call(**big, ws=P(0x10008), ws_bytes=need) == ERR_ALIGN
    assert call(**big, ws=FAKE, ws_bytes=need - 1) == ERR_WS


def test_logits_workspace(lib):
    q = lib.orpo_head_logits_q_workspace_bytes
    for bits in (4, 8):
        assert q(1, 2560, bits) == q(16, 3328, bits) == q(32, 1536, bits) == q(64, 768, bits) == q(1000, 768, bits) == 0
    for M, d, bits in ((17, 2048, 4), (64, 4096, 4), (16, 16384, 4), (1, 8200, 8), (1000, 4096, 4)):
        rows, seg = 16 if M <= 16 else 32 if M <= 32 else -(-M // 64) * 64, 1024 // bits
        assert q(M, d, bits) == rows * -(-d // seg) * seg * 2
    assert q(0, 256, 4) == q(4, 256, 5) == q(4, 4, 4) == 0


def test_select_host_checks(lib):
    def call(x=FAKE, ld=1000, bf16=0, score=FAKE, fin=None, eos=-1, batch=2, beams=4, V=1000, n=8, os=FAKE, op=FAKE,
             ot=FAKE, ws=FAKE, ws_bytes=1 << 30, st=FAKE):
        return lib.orpo_beam_select(x, ld, bf16, score, fin, eos, batch, beams, V, n, os, op, ot, None, ws, ws_bytes,
                                    st, None)

    assert call(batch=0) == OK
    for bad in (dict(batch=-1), dict(beams=0), dict(beams=65), dict(n=0), dict(n=65), dict(V=0), dict(V=7, n=8),
                dict(V=MAX_ROWS + 1, ld=MAX_ROWS + 1), dict(ld=999), dict(batch=1 << 19, beams=4)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in ("x", "score", "os", "op", "ot", "ws", "st"):
        assert call(**{bad: None}) == ERR_NULL, bad
    for bad in (dict(eos=-2), dict(eos=1000), dict(fin=FAKE, eos=-1)):
        assert call(**bad) == ERR_ARG, bad
    for bad in (dict(ws=P(0x10004)), dict(x=P(0x10002)), dict(x=P(0x10001), bf16=1), dict(score=P(0x10002))):
        assert call(**bad) == ERR_ALIGN, bad
    need = lib.orpo_beam_select_workspace_bytes(2, 4, 1000, 8)
    assert call(ws_bytes=need - 1) == ERR_WS


def test_select_workspace_stays_under_its_documented_bound(lib):
    for batch, beams, V, n in ((1, 1, 1, 1), (1, 4, 4096, 4), (4, 4, 262144, 8), (32, 8, 128256, 16), (7, 64, 50257, 64),
                               (1, 64, MAX_ROWS, 64), (1 << 14, 64, 1025, 1)):
        need = lib.orpo_beam_select_workspace_bytes(batch, beams, V, n)
        assert 0 < need <= 16 * batch * beams * (n + 1) * -(-V // 1024) + 4096
    assert lib.orpo_beam_select_workspace_bytes(-1, 4, 100, 4) == 0
    assert lib.orpo_beam_select_workspace_bytes(1, 4, 100, 101) == 0


def test_reorder_host_checks(lib):
    def call(state=FAKE, parent=FAKE, ld=4, length=FAKE, outer=2, batch=3, beams=4, rows=2, cap=16, unit=64, st=FAKE):
        return lib.orpo_beam_reorder(state, parent, ld, length, outer, batch, beams, rows, cap, unit, st, None)

    for empty in ("outer", "batch", "rows", "cap", "unit"):
        assert call(**{empty: 0}) == OK, empty
    for bad in (dict(outer=-1), dict(batch=-1), dict(beams=0), dict(beams=65, ld=65), dict(rows=-1), dict(cap=-1),
                dict(unit=-1), dict(ld=3), dict(outer=1 << 40, cap=1 << 40), dict(batch=1 << 31)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in ("state", "parent", "st"):
        assert call(**{bad: None}) == ERR_NULL, bad
    for bad in (dict(parent=P(0x10002)), dict(length=P(0x10001))):
        assert call(**bad) == ERR_ALIGN, bad


def test_parent_status_text(lib):
    assert "parent" in orpo.orpo_status_string(orpo.STATUS_BITS["parent"])


def test_python_entry_points_refuse_host_tensors(lib):
    t = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        orpo.orpo_head_logits_q(t.bfloat16(), t, t, t, 4, 32, 0.0, t, t)
    with pytest.raises(ValueError):
        orpo.orpo_beam_select(t, t[:, 0], None, -1, 2, t[:1, :2], t, t, None, t, t)
    with pytest.raises(ValueError):
        orpo.orpo_beam_reorder(t, t, None, t)
