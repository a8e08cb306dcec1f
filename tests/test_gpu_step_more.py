"""BeamDecoder.step with entries that get no new position: those that ended and let go of their pages, and those whose table is
full."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
import workloads
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

V, D = 4096, 256


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


@pytest.fixture(scope="module")
def weights():
    w = workloads.make("tiny")
    wq, s, b = workloads.quantize_affine(w.W, 4, 64)
    t16 = lambda a: torch.from_numpy(a.view(np.int16)).to(dev()).view(torch.bfloat16)  # noqa: E731
    return torch.from_numpy(wq).to(dev()), t16(s), t16(b)


def decoder(batch, beams, columns, n_pages, page, length):
    """A decoder whose beams have pages of their own for `length` positions."""
    dec = orpo.BeamDecoder(batch, beams, V, D, device=dev())
    pages = orpo.PagedStates(batch, beams, columns, n_pages, page, most=columns * page, status=dec.status, device=dev())
    pages.advance(torch.zeros_like(length), more=length, most=columns * page)
    dec.score.copy_(torch.arange(batch * beams, device=dev()).view(batch, beams) * -0.25)
    return dec, pages


def hidden(batch, beams, seed):
    return torch.randn((batch * beams, D), generator=torch.Generator("cuda").manual_seed(seed), device=dev()).bfloat16()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("raised", [False, True])
def test_no_page_goes_to_an_entry_that_was_released(weights, captured, raised):
    """As many free pages as the entries that are left need: had the other one taken any, they would not be enough."""
    batch, beams, page, columns, steps = 3, 4, 2, 12, 9
    length = t32([5, 6, 3])
    # the entries that are left end with at most ceil(15 / 2) and ceil(12 / 2) pages a beam
    dec, pages = decoder(batch, beams, columns, beams * (8 + 6), page, length)
    pool = torch.zeros((1, pages.pages, 1, page, 8), device=dev())
    pages.release(torch.tensor([0, 1, 0], dtype=torch.uint8, device=dev()))
    more, h = t32([1, 0, 1]), hidden(batch, beams, 0)
    step = lambda: dec.step(h, *weights, length=length, pages=pages, pools=(pool,), more=more)  # noqa: E731
    table, refs = pages.table.cpu().numpy(), pages.refs.cpu().numpy()
    assert (table[beams:2 * beams] == -1).all()
    if captured:
        keep = [t.clone() for t in (pages.table, pages.refs, dec.score, pool)]
        step()  # sets the device up
        for t, k in zip((pages.table, pages.refs, dec.score, pool), keep):
            t.copy_(k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for i in range(steps):
        h.copy_(hidden(batch, beams, i))
        n = length.cpu().numpy()
        graph.replay() if captured else step()
        table, refs, _, full = oracle.pages_advance(table, refs, page, dec.parent.cpu().numpy(), n, [1, 0, 1], 1)
        assert not full and int(dec.status) == 0
        assert np.array_equal(pages.table.cpu().numpy(), table) and np.array_equal(pages.refs.cpu().numpy(), refs)
        assert (table[beams:2 * beams] == -1).all()
        length += t32([1, 1 if raised else 0, 1])


def test_no_pools_by_either_name(weights):
    for kw in (dict(pools=None), dict(pools=()), {}):
        dec, pages = decoder(1, 3, 4, 20, 4, t32([5]))
        dec.step(hidden(1, 3, 0), *weights, **kw)
        dec.step(hidden(1, 3, 1), *weights, length=t32([5]), pages=pages, **kw)
        assert int(dec.status) == 0


def test_the_last_step_of_a_full_table(weights):
    """All positions are in use: the beams still follow their parents, and nothing is asked for."""
    batch, beams, page, columns = 2, 3, 4, 5
    length = t32([columns * page, 7])
    dec, pages = decoder(batch, beams, columns, 60, page, length)
    table, refs, n = pages.table.cpu().numpy(), pages.refs.cpu().numpy(), length.cpu().numpy()
    for i, more in enumerate(([0, 1], [0, 0])):
        parent, _ = dec.step(hidden(batch, beams, i), *weights, length=length, pages=pages, more=t32(more))
        table, refs, _, _ = oracle.pages_advance(table, refs, page, parent.cpu().numpy(), n, more, 1)
        assert int(dec.status) == 0
        assert np.array_equal(pages.table.cpu().numpy(), table) and np.array_equal(pages.refs.cpu().numpy(), refs)
    # what is asked for without `more` does not fit, and is reported
    dec.step(hidden(batch, beams, 9), *weights, length=length, pages=pages)
    assert int(dec.status) == orpo.STATUS_BITS["parent"]
