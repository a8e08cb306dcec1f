"""The calls behind the logits on a stream of their own while the current one is busy: their results are there, on that stream,
long before the current one gets to anything."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu

BATCH, BEAMS, PAGE, COLUMNS, PAGES, CAP, V = 3, 4, 4, 6, 90, 24, 5000


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


class Call:
    """One entry point on its buffers: run(stream), the buffers it writes, and what is in them afterwards."""

    def __init__(self, run, buffers, want):
        self.run, self.buffers, self.want = run, buffers, want
        self.before = [b.clone() for b in buffers]
        self.after = [torch.empty_like(b) for b in buffers]


def calls(seed):
    rng = np.random.default_rng(seed)
    rows = BATCH * BEAMS
    length = np.array([9, 16, 7])
    parent = rng.permuted(np.tile(np.arange(BEAMS), (BATCH, 1)), axis=1)
    parent[:, 0] = parent[:, 1]  # one beam twice, so that pages are copied
    token = rng.integers(0, V, (BATCH, BEAMS))
    history = rng.integers(0, V, (rows, CAP)).astype(np.int32)
    table = np.full((rows, COLUMNS), -1, dtype=np.int32)
    numbers = iter(rng.permutation(PAGES).tolist())
    for r in range(rows):
        for c in range(-(-int(length[r // BEAMS]) // PAGE)):
            table[r, c] = next(numbers)
    refs = oracle.holders(table, PAGES)
    st = status_tensor()
    dl, dp, dt, dh = t32(length), t32(parent), t32(token), t32(history)

    logits = rng.standard_normal((rows, V)).astype(np.float32)
    x = torch.from_numpy(logits).to(dev())
    yield "adjust", Call(lambda s: orpo.orpo_logits_adjust(x, BEAMS, st, dh, dl, repetition=1.25, no_repeat=1, stream=s), [x],
                         [oracle.logits_adjust(logits, BEAMS, history, length, repetition=1.25, no_repeat=1)[0].astype(np.float32)])
    h = t32(history)
    yield "history", Call(lambda s: orpo.orpo_beam_history(h, dp, dt, dl, st, stream=s), [h], [oracle.beam_history(history, parent, token, length)])

    def buffers():
        return (t32(table), t32(refs), torch.full((PAGES, 3), -9, dtype=torch.int32, device=dev()), t32([-9]),
                torch.empty(orpo.orpo_pages_workspace_bytes(rows, PAGES, PAGE, 1), dtype=torch.uint8, device=dev()))

    t, r, m, n, ws = buffers()
    wt, wr, wm, _ = oracle.pages_advance(table, refs, PAGE, parent, length, None, 1)
    assert wm
    yield "advance", Call(lambda s: orpo.orpo_pages_advance(t, r, PAGE, dp, dl, None, 1, m, n, ws, st, stream=s), [t, r, n], [wt, wr, [len(wm)]])
    pool = rng.integers(0, 256, (2, PAGES, 3, PAGE, 40)).astype(np.uint8)
    p, put, many = torch.from_numpy(pool).to(dev()), t32(wm), t32([len(wm)])
    yield "copy", Call(lambda s: orpo.orpo_pages_copy(p, put, many, st, stream=s), [p], [oracle.pages_copy(pool, wm)])
    t2, r2 = t32(table), t32(refs)
    ended = torch.tensor([1, 0, 1], dtype=torch.uint8, device=dev())
    yield "release", Call(lambda s: orpo.orpo_pages_release(t2, r2, ended, st, stream=s), [t2, r2], oracle.pages_release(table, refs, [1, 0, 1], BEAMS))
    t3, r3, m3, n3, ws3 = buffers()
    live = t32([-9])
    ct, cr, cl, cm = oracle.pages_compact(table, refs, PAGE)
    assert cm
    yield "compact", Call(lambda s: orpo.orpo_pages_compact(t3, r3, PAGE, t3, r3, live, m3, n3, ws3, st, stream=s), [t3, r3, live, n3], [ct, cr, [cl], [len(cm)]])


@pytest.mark.parametrize("name", ["adjust", "history", "advance", "copy", "release", "compact"])
def test_results_come_from_the_stream_that_was_asked_for(name):
    side = torch.cuda.Stream()
    call = dict(calls(1))[name]
    call.run(side)  # loads the kernels
    torch.cuda.synchronize()
    for b, old in zip(call.buffers, call.before):
        b.copy_(old)
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    torch.cuda._sleep(1_000_000_000)  # about half a second
    done.record()
    call.run(side)
    with torch.cuda.stream(side):
        for b, to in zip(call.buffers, call.after):
            to.copy_(b)
    side.synchronize()
    assert not done.query()  # the current stream has not come to anything behind the pause
    torch.cuda.synchronize()
    for to, want in zip(call.after, call.want):
        assert np.array_equal(to.cpu().numpy(), np.asarray(want))


def test_paged_states_on_a_stream_of_their_own():
    """advance, release and compact of PagedStates, their copies included, one behind the other on the side stream."""
    rng = np.random.default_rng(5)
    side, length = torch.cuda.Stream(), np.array([9, 16, 7])
    parent = np.tile([1, 1, 0, 3], (BATCH, 1))
    dp, dl, ended = t32(parent), t32(length), torch.tensor([0, 1, 0], dtype=torch.uint8, device=dev())
    data = rng.integers(0, 256, (2, PAGES, 3, PAGE, 40)).astype(np.uint8)
    zeros, st = t32([0] * BATCH), status_tensor()
    wait = 0
    for _ in range(2):  # the first time for loading the kernels
        pages = orpo.PagedStates(BATCH, BEAMS, COLUMNS, PAGES, PAGE, most=16, status=st, device=dev())
        pool = torch.from_numpy(data).to(dev())
        after = [torch.empty_like(x) for x in (pages.table, pages.refs, pool)]
        torch.cuda.synchronize()
        done = torch.cuda.Event()
        torch.cuda._sleep(1 + wait)
        done.record()
        pages.advance(zeros, more=dl, most=16, pools=(pool,), stream=side)
        pages.advance(dl, dp, pools=(pool,), stream=side)
        pages.release(ended, stream=side)
        pages.compact((pool,), stream=side)
        with torch.cuda.stream(side):
            for to, x in zip(after, (pages.table, pages.refs, pool)):
                to.copy_(x)
        side.synchronize()
        early = not done.query()
        torch.cuda.synchronize()
        wait = 1_000_000_000
    assert early and int(st) == 0
    table, refs, _, _ = oracle.pages_advance(np.full((BATCH * BEAMS, COLUMNS), -1, dtype=np.int32), np.zeros(PAGES, dtype=np.int32), PAGE, None, [0] * BATCH,
                                             length, 16)
    table, refs, moves, _ = oracle.pages_advance(table, refs, PAGE, parent, length, None, 1)
    assert moves
    want = oracle.pages_copy(data, moves)
    table, refs = oracle.pages_release(table, refs, [0, 1, 0], BEAMS)
    table, refs, _, moves = oracle.pages_compact(table, refs, PAGE)
    assert moves
    want = oracle.pages_copy(want, moves)
    for to, x in zip(after, (table, refs, want)):
        assert np.array_equal(to.cpu().numpy(), x)
