"""The entry points of orpo_pages.h against the oracle, which takes rows, columns and pages one at a time."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu

PARENT, PAGE, FULL = (orpo.STATUS_BITS[k] for k in ("parent", "page", "full"))


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def n32(t):
    return t.cpu().numpy()


class Pages:
    """A table and its counts of holders on the device, with what the calls need beside them."""

    def __init__(self, table, pages, page, most=1, pad=0, refs=None):
        self.rows, self.page = table.shape[0], page
        self.wide = torch.full((self.rows, table.shape[1] + pad), -9, dtype=torch.int32, device=dev())
        self.table = self.wide[:, :table.shape[1]]
        self.table.copy_(t32(table))
        self.refs = t32(oracle.holders(table, pages) if refs is None else refs)
        self.moves = torch.full((max(self.rows, pages // 2), 3), -9, dtype=torch.int32, device=dev())
        self.n = torch.full((1,), -9, dtype=torch.int32, device=dev())
        need = orpo.orpo_pages_workspace_bytes(self.rows, pages, page, most)
        self.guard = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=dev())
        self.ws, self.status = self.guard[:need], status_tensor()

    def advance(self, parent, length, more=None, most=1):
        orpo.orpo_pages_advance(self.table, self.refs, self.page, None if parent is None else t32(parent), t32(length),
                                None if more is None else t32(more), most, self.moves, self.n, self.ws, self.status)
        return self.state()

    def state(self):
        torch.cuda.synchronize()
        assert bool((self.guard[len(self.ws):] == 0xA5).all())
        assert bool((self.wide[:, self.table.shape[1]:] == -9).all())
        n = int(self.n.item())
        return n32(self.table), n32(self.refs), [tuple(m) for m in n32(self.moves)[:max(n, 0)].tolist()]


def same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(np.asarray(g), np.asarray(w)), (g, w)


def beams_table(rng, batch, beams, columns, pages, page, lengths, shared=0.5):
    """Beams that share the first part of their past, on random pages."""
    order = rng.permutation(pages).tolist()
    table = np.full((batch * beams, columns), -1, dtype=np.int32)
    for b in range(batch):
        n = -(-int(lengths[b]) // page)
        s = int(shared * (lengths[b] // page))
        common = [order.pop() for _ in range(s)]
        for k in range(beams):
            table[b * beams + k, :n] = common + [order.pop() for _ in range(n - s)]
    return table


@pytest.mark.parametrize("batch,beams,page,longest", [(1, 1, 1, 9), (1, 4, 16, 100), (3, 4, 5, 60), (2, 8, 16, 2500), (4, 9, 7, 80), (1, 17, 3, 40),
                                                      (1, 64, 4, 50), (70, 16, 8, 30), (1, 4, 1, 5000), (2, 6, 1, 2200)])
@pytest.mark.parametrize("more_pages", [0, 33000, 140000])
def test_decode_steps_against_the_oracle(batch, beams, page, longest, more_pages):
    """Several steps in a row, with new parents each and one more position each, in small and in large pools."""
    rng = np.random.default_rng(batch + beams + page)
    steps = 4
    lengths = rng.integers(0, longest, batch)
    lengths[0] = longest
    if batch > 1:
        lengths[1] = page * 2  # a border
    columns = -(-(longest + steps) // page)
    pages = batch * beams * (columns + 1) + 7 + more_pages
    table = beams_table(rng, batch, beams, columns, pages, page, lengths)
    p = Pages(table, pages, page, pad=3)
    want = table, oracle.holders(table, pages)
    for step in range(steps):
        parent = rng.integers(0, beams, (batch, beams)) if step != 2 else np.tile(np.arange(beams), (batch, 1))
        *want, full = oracle.pages_advance(*want[:2], page, parent, lengths, None, 1)
        same(p.advance(parent, lengths), want)
        assert not full and int(p.status.item()) == 0
        assert np.array_equal(want[1], oracle.holders(want[0], pages))
        lengths = lengths + 1


@pytest.mark.parametrize("batch,beams,page,most", [(1, 1, 16, 100), (5, 1, 4, 33), (3, 4, 7, 20), (40, 1, 3, 200), (1, 1, 1, 5000), (300, 2, 16, 90), (150, 2, 16, 90), (4096, 1, 8, 1), (4097, 1, 8, 1)])
def test_prompts_against_the_oracle(batch, beams, page, most):
    """Different numbers of new positions, none among them, on rows that have pages or none, and pages asked for before."""
    rng = np.random.default_rng(most)
    lengths = rng.integers(0, 50, batch) * rng.integers(0, 2, batch)
    more = rng.integers(0, most + 1, batch)
    more[-1], lengths[-1] = most, 0
    if batch > 2:
        more[0] = 0
    columns = -(-(50 + 2 * most) // page)
    pages = batch * beams * columns + 5
    table = beams_table(rng, batch, beams, columns, pages, page, lengths)
    p = Pages(table, pages, page, most=most)
    want = table, oracle.holders(table, pages)
    for m in (more, more, None):  # the second time nothing is missing
        *want, full = oracle.pages_advance(*want[:2], page, None, lengths, m, most)
        same(p.advance(None, lengths, m, most), want)
        assert not full and int(p.status.item()) == 0


@pytest.mark.parametrize("times,pages", [(1, 40), (1, 140000), (300, 40000), (1100, 40000)])
def test_pages_shared_between_entries_and_within_the_written_range(times, pages):
    """Rows of different entries that hold the same pages: all but the last, and all where something else holds it too, copy."""
    table = np.array([[0, 1, 2, -1], [0, 1, 2, -1], [0, 1, 2, -1], [3, 2, 1, -1], [2, 2, 2, -1]] * times, dtype=np.int32)
    for lengths, more in (([5, 6, 9, 4, 12], None), ([2, 2, 2, 0, 12], [10, 10, 10, 12, 1]), ([12] * 5, [4] * 5), ([0] * 5, [12] * 5)):
        lengths, more, most = lengths * times, more and more * times, 12 if more else 1
        p = Pages(table, pages, 4, most=most)
        want = oracle.pages_advance(table, oracle.holders(table, pages), 4, None, lengths, more, most)
        same(p.advance(None, lengths, more, most), want[:3])
        assert not want[3] and int(p.status.item()) == 0


def test_fork_alone_and_reserved_pages_stay():
    """most = 0 copies tables alone; pages behind ceil(length / page) are each beam's own."""
    table = np.array([[0, 1, 2], [0, 3, 4], [5, 6, -1], [7, 8, 9]], dtype=np.int32)
    p = Pages(table, 12, 4, most=0)
    want = oracle.pages_advance(table, oracle.holders(table, 12), 4, np.array([[1, 1], [1, 0]]), [5, 4], None, 0)
    same(p.advance([[1, 1], [1, 0]], [5, 4], None, 0), want[:3])
    assert want[0].tolist() == [[0, 3, 2], [0, 3, 4], [7, 6, -1], [5, 8, 9]]


def test_too_few_pages_change_nothing_but_the_fork():
    # one free page would do for one row, not for two
    t = np.array([[0, 1, -1], [0, 2, -1]], dtype=np.int32)
    p = Pages(t, 4, 4)
    want = oracle.pages_advance(t, oracle.holders(t, 4), 4, np.array([[1, 0]]), [8], None, 1)
    same(p.advance([[1, 0]], [8]), want[:3])
    assert want[3] and want[0].tolist() == [[0, 2, -1], [0, 1, -1]] and int(p.status.item()) == FULL and int(p.n.item()) == 0
    # after room is made, without parents
    p.refs = torch.cat((p.refs, p.refs.new_zeros(1)))
    p.ws = torch.empty(orpo.orpo_pages_workspace_bytes(2, 5, 4, 1), dtype=torch.uint8, device=dev())
    p.guard = p.ws
    p.status.zero_()
    got = p.advance(None, [8])
    assert got[0].tolist() == [[0, 2, 3], [0, 1, 4]] and int(p.status.item()) == 0


@pytest.mark.parametrize("rows,columns", [(3, 5461), (1200, 25), (1200, 4), (1000, 6), (5000, 2), (5, 30000)])
def test_too_few_pages_of_a_large_pool(rows, columns):
    """One page fewer than rows is free; it is enough for all but one."""
    held = rows * columns
    pages = held + rows - 1
    table = np.full((rows, columns + 1), -1, dtype=np.int32)
    table[:, :-1] = np.random.default_rng(rows).permutation(pages)[:held].reshape(rows, columns)
    refs = oracle.holders(table, pages)
    length = np.full(rows, 2 * columns)
    p = Pages(table, pages, 2, refs=refs)
    got = p.advance(None, length)
    assert int(p.status.item()) == FULL and int(p.n.item()) == 0
    assert np.array_equal(got[0], table) and np.array_equal(got[1], refs)
    p.status.zero_()
    more = np.ones(rows, dtype=np.int32)
    more[1] = 0
    want = oracle.pages_advance(table, refs, 2, None, length, more, 1)
    same(p.advance(None, length, more), want[:3])
    assert int(p.status.item()) == 0 and not want[3]


@pytest.mark.parametrize("columns,pages", [(5000, 6000), (3, 20000), (3, 140000), (5000, 140000)])
def test_wrong_entries_beside_right_ones_in_every_form(columns, pages):
    table = np.full((8, columns), -1, dtype=np.int32)
    table[:, :2] = np.arange(16).reshape(8, 2)
    p = Pages(table, pages, 4)
    got = p.advance([[1, 0], [1, 2], [0, 0], [1, 1]], [8, 8, 4 * columns, 6])
    want = oracle.pages_advance(table, oracle.holders(table, pages), 4, np.array([[1, 0], [0, 1], [0, 1], [1, 1]]), [8, 7, 7, 6], None, 1)
    assert int(p.status.item()) == PARENT
    same(got, want[:3])
    assert got[2] == [(15, 16, 2)]


def test_wrong_entries_are_left_as_they_are():
    table = np.arange(24, dtype=np.int32).reshape(12, 2)
    first = Pages(table, 60, 4, most=3)
    parents = [[1, 0], [0, 2], [-1, 0], [1, 0], [1, 0], [1, 0]]
    got = first.advance(parents, [4, 4, 4, -1, 9, 4], [1, 1, 1, 1, 0, 4], 3)
    assert int(first.status.item()) == PARENT
    assert np.array_equal(got[0][2:], table[2:]) and got[0][:2].tolist() == [[2, 1], [0, 3]] and got[2] == []
    p = Pages(table, 60, 4, most=3)
    got = p.advance(None, [5, 9, 6, -1, 8, 4], [1, 0, -1, 1, 1, 3], 3)
    assert int(p.status.item()) == PARENT and np.array_equal(got[0], table)


def test_page_numbers_out_of_range_are_reported_and_never_used():
    table = np.array([[0, 99], [-5, 1], [2**31 - 1, 2], [-2**31, 3]], dtype=np.int32)
    p = Pages(table, 10, 4, refs=[1, 1, 1, 1, 0, 0, 0, 0, 0, 0])
    got = p.advance([[1, 0], [1, 0]], [5, 3])
    assert int(p.status.item()) == PAGE
    assert got[0].tolist() == [[-5, 1], [0, 99], [-2**31, 2], [2**31 - 1, 3]] and got[2] == []
    p = Pages(table, 10, 4, refs=[1, 1, 1, 1, 0, 0, 0, 0, 0, 0])
    orpo.orpo_pages_release(p.table, p.refs, None, p.status)
    assert int(p.status.item()) == PAGE and bool((p.table == -1).all()) and int(p.refs.abs().sum()) == 0
    p = Pages(table, 10, 4, refs=[1, 1, 1, 1, 0, 0, 0, 0, 0, 0])
    live = torch.zeros(1, dtype=torch.int32, device=dev())
    orpo.orpo_pages_compact(p.table, p.refs, 4, p.table, p.refs, live, p.moves, p.n, p.ws, p.status)
    assert int(p.status.item()) == PAGE and np.array_equal(n32(p.table), table) and int(live.item()) == 4


def test_counts_that_are_too_low_are_reported():
    p = Pages(np.array([[3, 3], [3, -1]], dtype=np.int32), 5, 4, refs=[0, 0, 0, 2, 0])
    orpo.orpo_pages_release(p.table, p.refs, None, p.status)
    assert int(p.status.item()) == PAGE and p.refs.tolist() == [0] * 5
    p = Pages(np.array([[3, 0]], dtype=np.int32), 5, 4, refs=[1, 0, 0, 0, 0])
    live = torch.zeros(1, dtype=torch.int32, device=dev())
    orpo.orpo_pages_compact(p.table, p.refs, 4, p.table, p.refs, live, p.moves, p.n, p.ws, p.status)
    assert int(p.status.item()) == PAGE and p.table.tolist() == [[3, 0]]


@pytest.mark.parametrize("beams,columns", [(1, 5), (4, 300), (3, 1)])
def test_release_against_the_oracle(beams, columns):
    rng = np.random.default_rng(columns)
    batch, pages = 9, 400
    table = rng.integers(-1, pages, (batch * beams, columns)).astype(np.int32)
    refs = oracle.holders(table, pages)
    for ended in (rng.integers(0, 2, batch), np.zeros(batch, dtype=int), None):
        p = Pages(table, pages, 4, pad=2)
        put = None if ended is None else torch.from_numpy(ended.astype(np.uint8)).to(dev())
        for _ in range(2):  # the second time there is nothing to let go of
            orpo.orpo_pages_release(p.table, p.refs, put, p.status)
            same(p.state()[:2], oracle.pages_release(table, refs, ended, beams) if ended is not None else oracle.pages_release(table, refs, None, 1))
        assert int(p.status.item()) == 0


@pytest.mark.parametrize("pages", [1, 2, 3, 31, 1024, 1025, 5000, 70001])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.7, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_against_the_oracle(pages, share, in_place):
    rng = np.random.default_rng(pages)
    used = rng.permutation(pages)[:int(round(share * pages))]
    rows, columns = 7, max(3, len(used) // 5)
    table = np.full(rows * columns, -1, dtype=np.int32)
    if len(used):
        at = rng.permutation(rows * columns)
        fill = np.concatenate((used, rng.choice(used, 3)))[:rows * columns]
        table[at[:len(fill)]] = fill
    table = table.reshape(rows, columns)
    refs = oracle.holders(table, pages)
    want = oracle.pages_compact(table, refs, 6)
    p = Pages(table, pages, 6, pad=0 if in_place else 1, most=0)
    live = torch.full((1,), -9, dtype=torch.int32, device=dev())
    new, new_refs = (p.table, p.refs) if in_place else (torch.full_like(p.table, -9), torch.full_like(p.refs, -9))
    orpo.orpo_pages_compact(p.table, p.refs, 6, new, new_refs, live, p.moves, p.n, p.ws, p.status)
    old_table, old_refs, moves = p.state()
    assert int(p.status.item()) == 0 and int(live.item()) == want[2]
    same((n32(new), n32(new_refs), moves), (want[0], want[1], want[3]))
    if not in_place:
        same((old_table, old_refs), (table, refs))


@pytest.mark.parametrize("shape,dtype", [((1, 3, 1, 1, 1), torch.uint8), ((3, 9, 2, 16, 64), torch.bfloat16), ((2, 9, 3, 7, 33), torch.bfloat16),
                                         ((2, 9, 3, 9, 36), torch.bfloat16), ((5, 9, 1, 5, 7), torch.uint8), ((2, 9, 4, 16, 66), torch.uint8),
                                         ((1, 9, 1, 3, 20001), torch.float32), ((40, 9, 8, 32, 128), torch.bfloat16), ((2, 9, 2, 4, 1000), torch.uint8)])
@pytest.mark.parametrize("off", [0, 1, 4, 8])
def test_copy_against_the_oracle(shape, dtype, off):
    """Pools and runs of every alignment; no, some and all positions of a page."""
    rng = np.random.default_rng(off)
    size = torch.tensor([], dtype=dtype).element_size()
    raw = torch.from_numpy(rng.integers(0, 256, int(np.prod(shape)) * size + 64).astype(np.uint8)).to(dev())
    off = off // size * size  # a pool starts on its own type's border
    view = raw[off:off + int(np.prod(shape)) * size]
    pool = view.view(dtype).view(shape) if off % size == 0 and raw.data_ptr() % size == 0 else None
    before = raw.cpu().numpy().copy()
    page = shape[3]
    moves = [(0, 1, page), (2, 0 if shape[1] == 3 else 4, max(page - 1, 0)), (0, 3, 1), (5, 6, 0), (2, 8, page // 2)]
    moves = [m for m in moves if max(m[:2]) < shape[1]] if shape[1] > 3 else [(0, 1, page)]
    put, st = t32(moves + [(0, 2, page)] * 4), status_tensor()
    orpo.orpo_pages_copy(pool, put, t32([len(moves)]), st)
    torch.cuda.synchronize()
    bytes_shape = (*shape[:4], shape[4] * size)
    want = before.copy()
    want[off:off + view.numel()] = oracle.pages_copy(before[off:off + view.numel()].reshape(bytes_shape), moves).ravel()
    assert np.array_equal(raw.cpu().numpy(), want) and int(st.item()) == 0


def test_copy_leaves_wrong_moves_out():
    pool = torch.arange(6, dtype=torch.float32, device=dev()).view(1, 6, 1, 1, 1).repeat(2, 1, 3, 4, 5).contiguous()
    first = pool.clone()
    st = status_tensor()
    bad = [(6, 0, 4), (-1, 0, 4), (0, 6, 4), (0, -1, 4), (0, 2, 5), (0, 2, -1), (3, 3, 4)]
    orpo.orpo_pages_copy(pool, t32(bad), t32([len(bad)]), st)
    assert int(st.item()) == PAGE and torch.equal(pool, first)
    for n in (-1, 8):
        st.zero_()
        orpo.orpo_pages_copy(pool, t32([(0, 1, 4)] * 7), t32([n]), st)
        assert int(st.item()) == PAGE and torch.equal(pool, first)
    st.zero_()
    orpo.orpo_pages_copy(pool, t32(bad + [(4, 5, 2)]), t32([8]), st)
    first[:, 5, :, :2] = 4
    assert int(st.item()) == PAGE and torch.equal(pool, first)


def test_copy_past_2_31_bytes():
    """Pages on both sides of 2^31 and 2^32 bytes of a pool of 6 GB."""
    pool = torch.zeros((3, 4000, 4, 32, 4096), dtype=torch.uint8, device=dev())
    for i, p in enumerate((5, 3990, 2048)):
        pool[:, p] = torch.arange(1 + i, 4 + i, dtype=torch.uint8, device=dev()).view(3, 1, 1, 1)
    st = status_tensor()
    orpo.orpo_pages_copy(pool, t32([(5, 3999, 32), (3990, 6, 32), (2048, 2049, 7)]), t32([3]), st)
    assert int(st.item()) == 0
    for src, dst, n in ((5, 3999, 32), (3990, 6, 32), (2048, 2049, 7)):
        assert torch.equal(pool[:, dst, :, :n], pool[:, src, :, :n])
    assert not bool(pool[:, 2049, :, 7:].any()) and not bool(pool[:, 3998].any()) and not bool(pool[:, 7].any())


def test_empty_calls():
    st, n = status_tensor(), torch.full((1,), 5, dtype=torch.int32, device=dev())
    none = torch.empty((0, 3), dtype=torch.int32, device=dev())
    refs, ws = torch.zeros(4, dtype=torch.int32, device=dev()), torch.empty(4096, dtype=torch.uint8, device=dev())
    orpo.orpo_pages_advance(none, refs, 4, None, t32([]), None, 1, none, n, ws, st)
    assert int(n.item()) == 0
    p = Pages(np.full((2, 3), -1), 4, 4)
    got = p.advance(None, [0, 0], [0, 0], 1)
    assert got[2] == [] and int(p.n.item()) == 0 and (got[0] == -1).all()
    live = torch.full((1,), 5, dtype=torch.int32, device=dev())
    orpo.orpo_pages_compact(torch.empty((0, 0), dtype=torch.int32, device=dev()), refs, 4, torch.empty((0, 0), dtype=torch.int32, device=dev()),
                            torch.zeros_like(refs), live, torch.empty((2, 3), dtype=torch.int32, device=dev()), n, ws, st)
    assert int(live.item()) == 0 and int(n.item()) == 0 and int(st.item()) == 0
