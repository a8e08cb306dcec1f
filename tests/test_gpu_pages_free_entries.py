"""orpo_pages_compact on tables that hold pages which their counts call free: each is copied as it is and reported, wherever it
lies, in every form of the plan."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu

PAGE = orpo.STATUS_BITS["page"]


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def compact(table, refs, in_place):
    pages = len(refs)
    t, r = t32(table), t32(refs)
    new, new_refs = (t, r) if in_place else (torch.full_like(t, -9), torch.full_like(r, -9))
    live, n, st = t32([-9]), t32([-9]), status_tensor()
    moves = torch.full((max(1, pages // 2), 3), -9, dtype=torch.int32, device=dev())
    ws = torch.empty(orpo.orpo_pages_workspace_bytes(table.shape[0], pages, 4, 0), dtype=torch.uint8, device=dev())
    orpo.orpo_pages_compact(t, r, 4, new, new_refs, live, moves, n, ws, st)
    torch.cuda.synchronize()
    return new.cpu().numpy(), new_refs.cpu().numpy(), int(live), [tuple(m) for m in moves[:int(n)].tolist()], int(st)


@pytest.mark.parametrize("in_place", [False, True])
def test_the_smallest_case(in_place):
    """Page 1 moves into page 0, which the table holds too."""
    got = compact(np.array([[0, 1]]), np.array([0, 1]), in_place)
    assert got[0].tolist() == [[0, 0]] and got[1].tolist() == [1, 0] and got[2:] == (1, [(1, 0, 4)], PAGE)


# one CTA with its lists in shared memory; a cluster that rewrites the table itself; the table by a kernel of its own,
# behind one CTA and behind the cluster
@pytest.mark.parametrize("pages,rows,columns", [(31, 3, 20), (4096, 7, 600), (9000, 5, 1800), (300, 4, 4000), (9000, 10, 8000)])
@pytest.mark.parametrize("where", ["first", "inside", "last", "above", "none"])
@pytest.mark.parametrize("in_place", [False, True])
def test_held_free_pages_are_reported(pages, rows, columns, where, in_place):
    rng = np.random.default_rng(pages + columns)
    used = np.sort(rng.permutation(np.arange(1, pages - 2))[:pages // 2])
    live = len(used)
    free = np.setdiff1d(np.arange(pages), used)
    below = free[free < live]
    held = {"first": [below[0]], "inside": [below[len(below) // 2]], "last": [below[-1]], "above": [free[-1]], "none": []}[where]
    assert below[0] == 0 and (where in ("above", "none") or held[0] < live)
    table = rng.choice(np.concatenate((used, [-1])), rows * columns)
    at = rng.permutation(rows * columns)
    table[at[:live]] = used
    refs = oracle.holders(table, pages)
    table[at[live:live + len(held)]] = held
    table = table.reshape(rows, columns)
    want = oracle.pages_compact(table, refs, 4)
    got = compact(table, refs, in_place)
    assert got[4] == (PAGE if held else 0)
    for e in held:
        assert e in got[0]
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2:4] == want[2:]
