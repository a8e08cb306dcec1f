"""The documented limit on the columns asked for at once, on both sides of its border, where rounding a row's columns up to
whole units would cross it."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from orpo_preference_loss_gb300 import build as orpo_build

P = lambda a: ctypes.c_void_p(a)  # noqa: E731
FAKE = P(0x10000)  # never dereferenced
MOST = 1 << 30     # rows * (ceil((most - 1) / page) + 1)


@pytest.fixture(scope="module")
def lib():
    orpo_build.build()
    return orpo.load()


def sizes():
    """(rows, page, most) with rows * width at most MOST, as near as it gets."""
    for page in (1, 16, 1000):
        for width in (1024, 1025, 1070, 3500, 99_991, 1_000_003):
            rows = min(MOST // width, 1 << 20)
            yield rows, page, (width - 1) * page + 1
    yield 300000, 1, 3500
    yield 1_000_000, 1, 1070


def width_of(page, most):
    return -(-(most - 1) // page) + 1


@pytest.mark.parametrize("rows,page,most", list(sizes()))
def test_both_sides_of_the_border(lib, rows, page, most):
    assert rows * width_of(page, most) <= MOST
    need = orpo.orpo_pages_workspace_bytes(rows, 5000, page, most)
    assert 0 < need <= 16 * 5000 + 64 * rows * (most // page + 2) + 4096

    def call(rows, most, ws_bytes):  # a workspace that is too small is looked at behind the sizes
        return lib.orpo_pages_advance(FAKE, 1, 1, FAKE, 5000, page, None, 0, FAKE, None, most, rows, 1, FAKE, rows, FAKE, FAKE, ws_bytes, FAKE, None)

    assert call(rows, most, 16) == 5
    more = most + page * (MOST // rows - width_of(page, most) + 1)  # one column per row too many
    assert rows * width_of(page, more) > MOST and more < 1 << 31
    assert orpo.orpo_pages_workspace_bytes(rows, 5000, page, more) == 0 and call(rows, more, 1 << 40) == 2


def test_a_workspace_serves_smaller_calls_too(lib):
    """PagedStates asks for its workspace once, for all of its calls."""
    rng = np.random.default_rng(0)
    for _ in range(3000):
        page, width = int(rng.integers(1, 40)), int(np.exp(rng.uniform(0, 14)))
        rows = max(1, min(1 << 20, int(MOST // width * rng.choice([1, 1, 0.999, 0.9, rng.random()]))))
        most = (width - 1) * page + 1
        need = orpo.orpo_pages_workspace_bytes(rows, 100, page, most)
        assert need > 0
        few, less = int(rng.integers(1, rows + 1)), int(rng.integers(0, most + 1))
        for r, m in ((few, most), (rows, less), (few, less), (rows - 1, most), (rows, max(most - page, 0))):
            assert orpo.orpo_pages_workspace_bytes(r, 100, page, m) <= need


@pytest.mark.gpu
@pytest.mark.parametrize("rows,most", [(1_000_000, 1070), (300_000, 3500)])
def test_near_the_border_against_the_oracle(lib, rows, most):
    """Rows of a few columns, of which some ask for pages, in a call that might ask for a billion."""
    rng = np.random.default_rng(rows)
    columns, held = 6, 40_000
    table = np.full((rows, columns), -1, dtype=np.int32)
    at = rng.permutation(rows)[:held]
    table[at, 0] = np.arange(held) // 2  # pairs share a page
    length = np.zeros(rows, dtype=np.int32)
    length[at] = 1
    more = np.zeros(rows, dtype=np.int32)
    some = rng.permutation(rows)[:rows // 20]
    more[some] = rng.integers(1, columns, len(some))
    more[-1], more[0] = columns - 1, 3
    overwrite = at[:500]  # from position 0 on, so that shared pages are let go of
    length[overwrite], more[overwrite] = 0, 2
    pages = 400_000
    refs = oracle.holders(table, pages)
    want = oracle.pages_advance(table, refs, 1, None, length, more, most)
    assert not want[3]
    dev = torch.device("cuda:0")
    t, r, n, st = (torch.from_numpy(a).to(dev) for a in (table, refs, np.array([-9], dtype=np.int32), np.zeros(1, dtype=np.int32)))
    moves = torch.full((rows, 3), -9, dtype=torch.int32, device=dev)
    need = orpo.orpo_pages_workspace_bytes(rows, pages, 1, most)
    guard = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=dev)
    orpo.orpo_pages_advance(t, r, 1, None, torch.from_numpy(length).to(dev), torch.from_numpy(more).to(dev), most, moves, n, guard[:need], st)
    assert int(st) == 0 and int(n) == len(want[2]) and bool((guard[need:] == 0xA5).all())
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(r.cpu().numpy(), want[1])
