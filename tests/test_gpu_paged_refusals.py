"""A call of PagedStates or BeamDecoder that is refused has changed nothing: tables, counts of holders, pools, scores, histories
and states are what they were."""

import numpy as np
import pytest
import torch

import orpo_preference_loss_gb300 as orpo
import workloads
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

BATCH, BEAMS, PAGE, COLUMNS, PAGES, V, D = 2, 3, 4, 6, 60, 4096, 256


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def pool(pages=PAGES, page=PAGE, unit=8, rows=2):
    g = torch.Generator("cuda").manual_seed(pages + page + unit)
    return torch.randn((2, pages, rows, page, unit), generator=g, device=dev())


def wrong_pools():
    return {"pages": pool(pages=PAGES + 1), "fewer pages": pool(pages=PAGES - 1), "page": pool(page=PAGE + 1), "rank": pool()[0],
            "a view": pool(unit=16)[..., :8], "transposed": pool(rows=PAGE).transpose(2, 3), "host": pool().cpu(),
            # page * unit bytes past orpo_pages_copy's limit
            "size": torch.empty((1, PAGES, 0, PAGE, 2**29), dtype=torch.uint8, device=dev())}


def populated():
    """Beams that share pages, a beam's pages let go of, copies and moves to be made at the next call."""
    pages = orpo.PagedStates(BATCH, BEAMS, COLUMNS, PAGES, PAGE, most=COLUMNS * PAGE, device=dev())
    length = t32([9, 6])
    pages.advance(torch.zeros_like(length), more=length, most=9)
    pages.advance(length, parent=t32([[1, 1, 0], [2, 0, 2]]), more=torch.zeros_like(length))
    pages.release(torch.tensor([1, 0], dtype=torch.uint8, device=dev()))
    pages.admit(torch.zeros_like(length), t32([13, 0]), 13)
    pages.advance(t32([13, 6]), parent=t32([[0, 0, 0], [0, 1, 2]]), more=torch.zeros_like(length))
    assert int(pages.status) == 0
    return pages


def kept(pages, *more):
    return [t.clone() for t in (pages.table, pages.refs, pages.status, *more)]


def unchanged(pages, before, *more):
    torch.cuda.synchronize()
    for t, b in zip((pages.table, pages.refs, pages.status, *more), before):
        assert torch.equal(t, b)


@pytest.mark.parametrize("kind", ["pages", "fewer pages", "page", "rank", "a view", "transposed", "host", "size"])
@pytest.mark.parametrize("call", ["advance", "admit", "compact"])
def test_a_wrong_pool_is_refused_before_anything_changes(kind, call):
    pages, good, wrong = populated(), pool(), wrong_pools()[kind]
    if kind != "host":
        assert wrong.is_cuda
    length, more = t32([13, 6]), t32([1, 1])
    calls = {"advance": lambda pools: pages.advance(length, parent=t32([[0, 1, 0], [1, 1, 0]]), pools=pools),
             "admit": lambda pools: pages.admit(length, more, 1, pools=pools), "compact": lambda pools: pages.compact(pools)}
    before = kept(pages, good)
    for pools in ((wrong,), (good, wrong), (wrong, good)):
        with pytest.raises(ValueError, match="pool"):
            calls[call](pools)
        unchanged(pages, before, good)
    # and with right ones it does what it would have done
    calls[call](iter((good, good.clone())))
    torch.cuda.synchronize()
    assert int(pages.status) == 0 and int(pages.n_moves) > 0 and not torch.equal(good, before[3])
    assert not torch.equal(pages.table, before[0])


@pytest.fixture(scope="module")
def weights():
    w = workloads.make("tiny")
    wq, s, b = workloads.quantize_affine(w.W, 4, 64)
    t16 = lambda a: torch.from_numpy(a.view(np.int16)).to(dev()).view(torch.bfloat16)  # noqa: E731
    return torch.from_numpy(wq).to(dev()), t16(s), t16(b)


STEP = ("pool", "second pool", "host pool", "pools without pages", "more without pages", "more of another type", "more of another size", "history of another type",
        "history of other rows", "empty history", "length of another type", "length of another size", "length on the host", "state", "second state",
        "state of other beams", "bias values alone", "bias tokens alone", "mask rows alone", "masks alone", "masks of another size")


@pytest.mark.parametrize("kind", STEP)
@pytest.mark.parametrize("penalties", [{}, dict(repetition=1.2)])
def test_a_wrong_step_is_refused_before_anything_changes(weights, kind, penalties):
    rows = BATCH * BEAMS
    dec = orpo.BeamDecoder(BATCH, BEAMS, V, D, device=dev(), eos=1, **penalties)
    pages, good, state = populated(), pool(), torch.randn((2, rows, 3, 20, 8), device=dev())
    history = torch.arange(rows * 20, dtype=torch.int32, device=dev()).view(rows, 20)
    h = torch.randn((rows, D), generator=torch.Generator("cuda").manual_seed(1), device=dev()).bfloat16()
    usual = dict(states=(state,), length=t32([13, 6]), history=history, pages=pages, pools=(good,))
    wrong = {"pool": dict(pools=(pool(page=5),)), "second pool": dict(pools=(good, good[..., :5])), "host pool": dict(pools=(good, good.cpu())),
             "pools without pages": dict(pages=None), "more without pages": dict(pages=None, pools=(), more=t32([1, 0])),
             "more of another type": dict(more=t32([1, 0]).long()), "more of another size": dict(more=t32([1])),
             "history of another type": dict(history=history.long()), "history of other rows": dict(history=history[:4]),
             "empty history": dict(history=history[:, :0]), "length of another type": dict(length=t32([13, 6]).long()), "length of another size": dict(length=t32([13])),
             "length on the host": dict(length=t32([13, 6]).cpu()), "state": dict(states=(state[0],)), "second state": dict(states=(state, state[..., :5])),
             "state of other beams": dict(states=(state[:, :4].contiguous(),)), "bias values alone": dict(bias_value=torch.zeros((BATCH, 4), device=dev())),
             "bias tokens alone": dict(bias_token=t32([[1, 2], [3, 4]])), "mask rows alone": dict(mask_row=t32([0] * rows)),
             "masks alone": dict(masks=t32([[0] * (V // 32)])), "masks of another size": dict(masks=t32([[0] * 5]), mask_row=t32([0] * rows))}[kind]
    held = (dec.score, dec.finished, dec.status, history, state, good)
    before = kept(pages, *held)
    with pytest.raises((ValueError, orpo.OrpoError)):
        dec.step(h, *weights, **{**usual, **wrong})
    unchanged(pages, before, *held)
    dec.step(h, *weights, **usual)
    torch.cuda.synchronize()
    assert int(dec.status) == int(pages.status) == 0 and not torch.equal(dec.score, before[3])
    assert not torch.equal(history, before[6])
