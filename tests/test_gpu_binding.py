"""csrc/binding.cpp and the way through ctypes: usual arguments take the first, and both give the same."""

import numpy as np
import pytest
import torch

import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def all_calls(stream=None):
    """Each of the calls once, with every optional argument, on strided rows; the buffers they wrote."""
    rng = np.random.default_rng(0)
    batch, beams, V, page, pages = 2, 3, 1000, 4, 50
    rows, st = batch * beams, status_tensor()
    x = torch.from_numpy(rng.standard_normal((rows, V + 5)).astype(np.float32)).to(dev())
    history = t32(rng.integers(0, V, (rows, 20)))
    length, prompt = t32([9, 5]), t32([2, 0])
    parent, token = t32([[1, 1, 0], [2, 0, 2]]), t32(rng.integers(0, V, (batch, beams)))
    bias = t32(rng.integers(0, V, (batch, 7))), torch.from_numpy(rng.standard_normal((batch, 7)).astype(np.float32)).to(dev())
    masks, mask_row = t32(rng.integers(-2**31, 2**31, (2, 32))), t32([0, 1, -1, 0, 1, -1])
    orpo.orpo_logits_adjust(x[:, :V], beams, st, history[:, :16], length, prompt, 1.2, 0.3, 0.1, 2, *bias, masks, mask_row, stream)
    one = x[:, :V].clone()
    orpo.orpo_logits_adjust(one, beams, st, bias_token=bias[0][0], bias_value=bias[1][0], stream=stream)
    orpo.orpo_beam_history(history[:, :16], parent, token, length, st, stream)
    wide = torch.full((rows, 11), -1, dtype=torch.int32, device=dev())
    refs, moves, n, live = torch.zeros(pages, dtype=torch.int32, device=dev()), torch.zeros((pages, 3), dtype=torch.int32, device=dev()), t32([0]), t32([0])
    ws = torch.empty(orpo.orpo_pages_workspace_bytes(rows, pages, page, 9), dtype=torch.uint8, device=dev())
    pool = torch.from_numpy(rng.integers(0, 256, (2, pages, 3, page, 24)).astype(np.uint8)).to(dev())
    orpo.orpo_pages_advance(wide[:, :8], refs, page, None, torch.zeros_like(length), length, 9, moves, n, ws, st, stream)
    orpo.orpo_pages_advance(wide[:, :8], refs, page, parent, length, None, 1, moves, n, ws, st, stream)
    orpo.orpo_pages_copy(pool, moves, n, st, stream)
    orpo.orpo_pages_release(wide[:, :8], refs, torch.tensor([True, False], device=dev()), st, stream)
    orpo.orpo_pages_release(wide[3:4, :8], refs, None, st, stream)
    new, new_refs = torch.full((rows, 9), -7, dtype=torch.int32, device=dev()), torch.empty_like(refs)
    orpo.orpo_pages_compact(wide[:, :8], refs, page, new[:, :8], new_refs, live, moves, n, ws, st, stream)
    orpo.orpo_pages_copy(pool, moves, n, st, stream)
    torch.cuda.synchronize()
    assert int(st) == 0 and int(n) > 0
    return [t.cpu() for t in (x, one, history, wide, refs, moves[:int(n)], n, new, new_refs, live, pool)]


class NoBinding:
    """Answers as the module of csrc/binding.cpp does to arguments that it does not take."""

    def __getattr__(self, name):
        return lambda *args: -1


@pytest.mark.parametrize("side", [False, True])
def test_usual_arguments_do_not_go_through_ctypes(monkeypatch, side):
    def looked_at(*tensors):
        raise AssertionError("the arguments were looked at one by one")

    assert type(orpo._bound()).__name__ == "module"
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    monkeypatch.setattr(orpo, "_here", looked_at)
    if side:
        with torch.cuda.stream(stream):
            all_calls(stream)
    else:
        all_calls()


def test_both_ways_give_the_same(monkeypatch):
    fast = all_calls()
    monkeypatch.setattr(orpo, "_fast", NoBinding())
    for a, b in zip(fast, all_calls()):
        assert torch.equal(a, b)


def test_whole_numbers_are_not_cut_to_their_c_types(monkeypatch):
    """2^32 + 2 is not 2, nor is 2^64 + 4 a page of 4 positions."""
    st, x = status_tensor(), torch.ones((2, 64), device=dev())
    history, length = torch.zeros((2, 8), dtype=torch.int32, device=dev()), t32([3])
    table, refs, moves, n = t32([[-1] * 3] * 2), t32([0] * 9), t32([[0] * 3] * 4), t32([0])
    ws = torch.zeros(4096, dtype=torch.uint8, device=dev())
    for fast in (orpo._bound(), NoBinding()):
        monkeypatch.setattr(orpo, "_fast", fast)
        for kw in (dict(no_repeat=2**32 + 2), dict(no_repeat=2**64), dict(no_repeat=-2**32 + 2), dict(beams=2**32 + 2)):
            with pytest.raises((ValueError, orpo.OrpoError)):
                orpo.orpo_logits_adjust(**{**dict(logits=x, beams=2, status=st, history=history, length=length), **kw})
        for kw in (dict(page=2**64 + 4), dict(most=2**64 + 1), dict(most=-2**64 + 1)):
            with pytest.raises((ValueError, orpo.OrpoError)):
                orpo.orpo_pages_advance(**{**dict(table=table, refs=refs, page=4, parent=None, length=length, more=None, most=1, moves=moves, n_moves=n,
                                                  workspace=ws, status=st), **kw})
        with pytest.raises((ValueError, orpo.OrpoError)):
            orpo.orpo_pages_compact(table, refs, 2**64 + 4, table.clone(), refs.clone(), t32([0]), moves, n, ws, st)
    for bad in ((2**64 + 2, 9, 4, 1), (2, 2**64 + 9, 4, 1), (2, 9, 2**64 + 4, 1), (2, 9, 4, 2**64 + 1)):
        with pytest.raises(ValueError):
            orpo.orpo_pages_workspace_bytes(*bad)
    torch.cuda.synchronize()
    assert bool((x == 1).all()) and bool((table == -1).all()) and int(st) == 0
