"""Host-side checks of the logits' adjustment, the histories and the shared pages: every refusal returns its code before any
CUDA call."""

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


def test_adjust_host_checks(lib):
    def call(x=FAKE, ld=1000, bf16=0, batch=2, beams=4, V=1000, h=FAKE, ld_h=64, cap=64, length=FAKE, prompt=None, rep=1.5, pres=0.0,
             freq=0.0, n=0, bt=None, bv=None, ld_b=0, nb=0, masks=None, ld_m=0, nm=0, row=None, st=FAKE):
        return lib.orpo_logits_adjust(x, ld, bf16, batch, beams, V, h, ld_h, cap, length, prompt, rep, pres, freq, n, bt, bv, ld_b, nb,
                                      masks, ld_m, nm, row, st, None)

    mask = dict(masks=FAKE, ld_m=32, nm=3, row=FAKE)
    bias = dict(bt=FAKE, bv=FAKE, nb=5)
    assert call(batch=0) == OK
    assert call(rep=1.0, h=None, length=None) == OK  # nothing to do
    assert call(h=None, length=None, cap=0) == OK
    for bad in (dict(batch=-1), dict(batch=(1 << 20) + 1), dict(beams=0), dict(beams=(1 << 20) + 1), dict(batch=1 << 18, beams=8), dict(V=0),
                dict(V=MAX_ROWS + 1, ld=MAX_ROWS + 1), dict(ld=999), dict(cap=-1), dict(cap=1 << 28, ld_h=1 << 28), dict(ld_h=63),
                {**bias, "nb": -1}, {**bias, "nb": 4097}, {**bias, "ld_b": 4}, {**mask, "nm": 0}, {**mask, "nm": 1 << 31},
                {**mask, "ld_m": 31}):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in (dict(rep=0.0), dict(rep=-1.0), dict(rep=math.nan), dict(rep=math.inf), dict(pres=math.nan), dict(freq=-math.inf),
                dict(n=-1), dict(n=33)):
        assert call(**bad) == ERR_ARG, bad
    for bad in (dict(x=None), dict(st=None), dict(h=None), dict(length=None), dict(h=None, rep=1.0, n=2), {**bias, "bt": None},
                {**bias, "bv": None}, {**mask, "row": None}, {**mask, "masks": None}):
        assert call(**bad) == ERR_NULL, bad
    for bad in (dict(x=P(0x10002)), dict(x=P(0x10001), bf16=1), dict(h=P(0x10002)), dict(length=P(0x10001)), dict(prompt=P(0x10003)),
                {**bias, "bt": P(0x10002)}, {**bias, "bv": P(0x10002)}, {**mask, "masks": P(0x10001)}, {**mask, "row": P(0x10002)},
                dict(st=P(0x10002))):
        assert call(**bad) == ERR_ALIGN, bad


def test_history_host_checks(lib):
    def call(h=FAKE, ld=64, cap=64, parent=FAKE, ld_p=4, token=FAKE, ld_t=4, length=FAKE, batch=2, beams=4, st=FAKE):
        return lib.orpo_beam_history(h, ld, cap, parent, ld_p, token, ld_t, length, batch, beams, st, None)

    assert call(batch=0) == OK
    for bad in (dict(batch=-1), dict(beams=0), dict(beams=65, ld_p=65, ld_t=65), dict(batch=1 << 15, beams=64, ld_p=64, ld_t=64),
                dict(cap=0), dict(cap=1 << 28, ld=1 << 28), dict(ld=63), dict(ld_p=3), dict(ld_t=3)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in ("h", "parent", "token", "length", "st"):
        assert call(**{bad: None}) == ERR_NULL, bad
        assert call(**{bad: P(0x10002)}) == ERR_ALIGN, bad


TABLE_LIMITS = (dict(pages=0), dict(pages=(1 << 24) + 1), dict(columns=-1), dict(columns=9))


def test_advance_host_checks(lib):
    need = orpo.orpo_pages_workspace_bytes(8, 100, 16, 1)

    def call(table=FAKE, ld=8, columns=8, refs=FAKE, pages=100, page=16, parent=FAKE, ld_p=4, length=FAKE, more=None, most=1, batch=2,
             beams=4, moves=FAKE, max_moves=8, n=FAKE, ws=FAKE, ws_bytes=need, st=FAKE):
        return lib.orpo_pages_advance(table, ld, columns, refs, pages, page, parent, ld_p, length, more, most, batch, beams, moves,
                                      max_moves, n, ws, ws_bytes, st, None)

    for bad in TABLE_LIMITS + (dict(batch=-1), dict(beams=0), dict(beams=65, ld_p=65, max_moves=999), dict(page=0), dict(page=(1 << 16) + 1),
                               dict(batch=1 << 19, max_moves=1 << 30), dict(page=1 << 16, columns=1 << 15, ld=1 << 15), dict(most=-1),
                               dict(most=1 << 31), dict(ld_p=3), dict(max_moves=7), dict(batch=1 << 18, max_moves=1 << 30, most=(1 << 31) - 1)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in ("table", "refs", "length", "moves", "n", "ws", "st"):
        assert call(**{bad: None}) == ERR_NULL, bad
    for bad in ("table", "refs", "parent", "length", "more", "moves", "n", "st"):
        assert call(**{bad: P(0x10002)}) == ERR_ALIGN, bad
    assert call(ws=P(0x10008)) == ERR_ALIGN
    assert call(ws_bytes=16) == ERR_WS


def test_copy_host_checks(lib):
    def call(pool=FAKE, outer=2, pages=10, rows=3, page=16, unit=64, moves=FAKE, max_moves=4, n=FAKE, st=FAKE):
        return lib.orpo_pages_copy(pool, outer, pages, rows, page, unit, moves, max_moves, n, st, None)

    for empty in ("outer", "rows", "unit", "max_moves"):
        assert call(**{empty: 0}) == OK, empty
    for bad in (dict(outer=-1), dict(pages=0), dict(pages=(1 << 24) + 1), dict(rows=-1), dict(page=0), dict(unit=-1), dict(max_moves=-1),
                dict(max_moves=1 << 31), dict(unit=1 << 28), dict(outer=1 << 40, rows=1 << 12), dict(outer=1 << 62)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in ("pool", "moves", "n", "st"):
        assert call(**{bad: None}) == ERR_NULL, bad
    for bad in ("moves", "n", "st"):
        assert call(**{bad: P(0x10002)}) == ERR_ALIGN, bad


def test_release_host_checks(lib):
    def call(table=FAKE, ld=8, columns=8, refs=FAKE, pages=100, ended=FAKE, batch=2, beams=4, st=FAKE):
        return lib.orpo_pages_release(table, ld, columns, refs, pages, ended, batch, beams, st, None)

    assert call(batch=0) == call(columns=0) == OK
    for bad in TABLE_LIMITS + (dict(batch=-1), dict(beams=0), dict(beams=65), dict(batch=1 << 20, beams=2)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in ("table", "refs", "st"):
        assert call(**{bad: None}) == ERR_NULL, bad
        assert call(**{bad: P(0x10002)}) == ERR_ALIGN, bad


def test_compact_host_checks(lib):
    need = orpo.orpo_pages_workspace_bytes(8, 100, 16, 0)

    def call(table=FAKE, ld=8, columns=8, rows=8, refs=FAKE, pages=100, page=16, new=P(0x20000), ld_new=8, new_refs=P(0x30000), live=FAKE,
             moves=FAKE, max_moves=50, n=FAKE, ws=FAKE, ws_bytes=need, st=FAKE):
        return lib.orpo_pages_compact(table, ld, columns, rows, refs, pages, page, new, ld_new, new_refs, live, moves, max_moves, n, ws,
                                      ws_bytes, st, None)

    for bad in TABLE_LIMITS + (dict(rows=-1), dict(rows=(1 << 20) + 1), dict(page=0), dict(ld_new=7), dict(max_moves=49),
                               dict(new=FAKE, ld_new=9)):
        assert call(**bad) == ERR_SHAPE, bad
    for bad in ("table", "refs", "new", "new_refs", "live", "moves", "n", "ws", "st"):
        assert call(**{bad: None}) == ERR_NULL, bad
    for bad in ("table", "refs", "new", "new_refs", "live", "moves", "n", "st"):
        assert call(**{bad: P(0x10002)}) == ERR_ALIGN, bad
    assert call(ws=P(0x10008)) == ERR_ALIGN
    assert call(ws_bytes=need // 4) == ERR_WS


def test_pages_workspace_stays_under_its_documented_bound(lib):
    for rows, pages, page, most in ((1, 1, 1, 1), (4, 27, 16, 1), (256, 163840, 16, 8192), (1 << 20, 1 << 24, 16, 1), (64, 4227, 32, 0),
                                    (8, 100, 1 << 16, 1 << 20), (0, 5, 7, 3), (3, 99, 1, 500)):
        need = orpo.orpo_pages_workspace_bytes(rows, pages, page, most)
        assert 0 < need <= 16 * pages + 64 * rows * (most // page + 2) + 4096
    for bad in ((-1, 5, 7, 3), (1, 0, 7, 3), (1, 5, 0, 3), (1, 5, 7, -1), ((1 << 20) + 1, 5, 7, 3), (1 << 20, 5, 1, 1 << 20)):
        assert orpo.orpo_pages_workspace_bytes(*bad) == 0


def test_status_texts(lib):
    for bit, text in (("page", "page"), ("full", "free pages"), ("mask", "mask")):
        assert text in orpo.orpo_status_string(orpo.STATUS_BITS[bit])
    every = orpo.orpo_status_string(sum(orpo.STATUS_BITS.values()))
    assert every.count("; ") == len(orpo.STATUS_BITS) - 1 and every.endswith("mask number out of range")


def test_python_entry_points_refuse_host_tensors(lib):
    t = torch.zeros((2, 64), dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        orpo.orpo_logits_adjust(t.float(), 2, one, t, one)
    with pytest.raises(ValueError):
        orpo.orpo_beam_history(t, t[:1, :2], t[:1, :2], one, one)
    with pytest.raises(ValueError):
        orpo.orpo_pages_advance(t, one, 16, None, one, None, 1, t[:, :3], one, one, one)
    with pytest.raises(ValueError):
        orpo.orpo_pages_copy(t.view(1, 2, 1, 16, 4), t[:, :3], one, one)
    with pytest.raises(ValueError):
        orpo.orpo_pages_release(t, one, None, one)
    with pytest.raises(ValueError):
        orpo.orpo_pages_compact(t, one, 16, t, one, one, t[:, :3], one, one, one)
