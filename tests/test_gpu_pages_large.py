"""Page plans at the upper end of their range: pools of hundreds of thousands of pages, where each warp has more pages than it
keeps in registers and several tiles, and more than a million columns asked for at once."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

FULL = orpo.STATUS_BITS["full"]


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def compacted(table, refs, page):
    """oracle.pages_compact in whole arrays: (table, refs, live, moves [n, 3])."""
    number = np.arange(len(refs))
    live = int((refs > 0).sum())
    holes, movers = number[(refs == 0) & (number < live)], number[(refs > 0) & (number >= live)]
    to = number.copy()
    to[movers] = holes
    new_refs = refs.copy()
    new_refs[holes], new_refs[movers] = refs[movers], 0
    return np.where(table < 0, table, to[np.maximum(table, 0)]), new_refs, live, np.stack((movers, holes, np.full(len(holes), page)), 1)


def random_table(rng, pages, rows, columns, used):
    """Every one of `used` random pages once, some of them again, -1 in the rest."""
    pick = rng.permutation(pages)[:used]
    table = np.full(rows * columns, -1, dtype=np.int32)
    again = min(len(pick), (table.size - used) // 2)
    table[rng.permutation(table.size)[:used + again]] = np.concatenate((pick, pick[:again]))
    return table.reshape(rows, columns)


@pytest.mark.parametrize("pages,used", [(1, 0), (1, 1), (7, 3), (50, 20), (50, 49), (64, 64), (333, 100)])
def test_the_whole_array_form_is_the_oracle(pages, used):
    table = random_table(np.random.default_rng(pages), pages, 6, 70, used)
    refs = oracle.holders(table, pages)
    got, want = compacted(table, refs, 5), oracle.pages_compact(table, refs, 5)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == want[2]
    assert [tuple(m) for m in got[3].tolist()] == want[3]


# the table is rewritten by the cluster (up to 65536 entries, so most pages are in no table) and by a kernel of its own
@pytest.mark.gpu
@pytest.mark.parametrize("pages,rows,columns", [(262144, 64, 5000), (262145, 64, 5000), (300001, 40, 1500), (300001, 64, 5000), (1000003, 256, 4200)])
@pytest.mark.parametrize("share", [0.03, 0.5, 0.97])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_of_large_pools(pages, rows, columns, share, in_place):
    rng = np.random.default_rng(pages + rows)
    used = min(int(share * pages), rows * columns)
    table = random_table(rng, pages, rows, columns, used)
    refs = oracle.holders(table, pages)
    want = compacted(table, refs, 16)
    t, r = t32(table), t32(refs)
    new, new_refs = (t, r) if in_place else (torch.full_like(t, -9), torch.full_like(r, -9))
    moves = torch.full((pages // 2, 3), -9, dtype=torch.int32, device=dev())
    live, n, st = t32([-9]), t32([-9]), status_tensor()
    ws = torch.empty(orpo.orpo_pages_workspace_bytes(rows, pages, 16, 0), dtype=torch.uint8, device=dev())
    orpo.orpo_pages_compact(t, r, 16, new, new_refs, live, moves, n, ws, st)
    assert int(st) == 0 and int(live) == want[2] and int(n) == len(want[3])
    assert np.array_equal(moves[:int(n)].cpu().numpy(), want[3]) and bool((moves[int(n):] == -9).all())
    assert np.array_equal(new.cpu().numpy(), want[0]) and np.array_equal(new_refs.cpu().numpy(), want[1])
    if not in_place:
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)


def advance(table, refs, page, parent, length, more, most):
    t, r = t32(table), t32(refs)
    moves, n, st = torch.full((len(table), 3), -9, dtype=torch.int32, device=dev()), t32([-9]), status_tensor()
    need = orpo.orpo_pages_workspace_bytes(len(table), len(refs), page, most)
    guard = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=dev())
    orpo.orpo_pages_advance(t, r, page, None if parent is None else t32(parent), t32(length), None if more is None else t32(more), most, moves, n,
                            guard[:need], st)
    assert bool((guard[need:] == 0xA5).all())
    return t.cpu().numpy(), r.cpu().numpy(), [tuple(m) for m in moves[:max(int(n), 0)].tolist()], int(st)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,page,most,spare", [(64, 1, 20000, 90000), (64, 1, 20000, -1), (400000, 4, 9, 9), (9000, 2, 260, 0)])
def test_more_than_a_million_columns_asked_for(rows, page, most, spare):
    """Long and short rows, among them rows that hold pages together; spare: free pages that are left, or one too few."""
    rng = np.random.default_rng(rows)
    width = (most + page - 2) // page + 1
    columns = width + 4
    length = rng.integers(0, 3 * page, rows).astype(np.int32)
    more = np.full(rows, most, dtype=np.int32)
    more[rng.integers(0, rows, rows // 8)] = 0
    table = np.full((rows, columns), -1, dtype=np.int32)
    held = rows * 3
    table[:, :3] = np.arange(held).reshape(rows, 3)
    table[1:rows // 2:3, :3] = table[0:rows // 2 - 1:3, :3][:len(table[1:rows // 2:3])]  # pairs of neighbours
    refs = oracle.holders(table, held)
    probe = oracle.pages_advance(table, np.concatenate((refs, np.zeros(rows * width, dtype=np.int32))), page, None, length, more, most)
    assert not probe[3]
    taken = int((probe[0] >= held).sum()) + int(((probe[0] < held) & (probe[0] >= 0) & (refs[np.clip(probe[0], 0, held - 1)] == 0)).sum())
    pages = held + taken + spare - int((refs == 0).sum())
    refs = np.concatenate((refs, np.zeros(pages - held, dtype=np.int32)))
    want = oracle.pages_advance(table, refs, page, None, length, more, most)
    assert want[3] == (spare < 0) and rows * width > 1 << 20
    got = advance(table, refs, page, None, length, more, most)
    assert got[3] == (FULL if spare < 0 else 0)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == want[2]


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [262145, 1000003])
@pytest.mark.parametrize("batch,beams", [(2, 4), (40, 12)])
def test_decode_steps_in_large_pools(pages, batch, beams):
    """The lowest free pages lie at the front, or behind hundreds of thousands of pages in use."""
    rng = np.random.default_rng(pages + batch)
    page, columns = 8, 40
    for low in (False, True):
        length = rng.integers(1, (columns - 2) * page, batch)
        table = np.full((batch * beams, columns), -1, dtype=np.int32)
        for r in range(batch * beams):
            n = -(-int(length[r // beams]) // page)
            table[r, :n] = rng.choice(pages, n, replace=False) if low else pages - 1 - r * columns - np.arange(n)
        refs = oracle.holders(table, pages)
        if not low:
            refs[:pages - batch * beams * columns - 5000] += 1  # held by others
        for _ in range(2):
            parent = rng.integers(0, beams, (batch, beams))
            want = oracle.pages_advance(table, refs, page, parent, length, None, 1)
            got = advance(table, refs, page, parent, length, None, 1)
            assert got[3] == 0 and not want[3]
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == want[2]
            table, refs = want[:2]
            length = length + 1
