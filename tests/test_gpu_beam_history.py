"""orpo_beam_history against the oracle: every kernel form, lengths at both ends, wrong parents and lengths."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu

PARENT = orpo.STATUS_BITS["parent"]


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


@pytest.mark.parametrize("pad,off", [(0, 0), (3, 0), (1, 1), (4, 2)])
@pytest.mark.parametrize("batch,beams,cap", [(1, 1, 1), (1, 4, 100), (3, 4, 1030), (2, 8, 513), (2, 9, 700), (1, 16, 64), (2, 17, 300), (1, 64, 129),
                                             (5, 3, 5000)])
def test_against_the_oracle(batch, beams, cap, pad, off):
    rng = np.random.default_rng(batch * beams + cap)
    for lengths in (rng.integers(0, cap, batch), np.zeros(batch, dtype=int), np.full(batch, cap - 1), np.full(batch, min(cap - 1, 6))):
        flat = torch.full((batch * beams * (cap + pad) + off,), -7, dtype=torch.int32, device=dev())
        h = flat[off:].view(batch * beams, cap + pad)
        h[:, :cap] = torch.from_numpy(rng.integers(0, 1000, (batch * beams, cap)).astype(np.int32)).to(dev())
        parent = rng.integers(0, beams, (batch, beams + 2)).astype(np.int32)
        token = rng.integers(0, 1000, (batch, beams + 1)).astype(np.int32)
        want = oracle.beam_history(h[:, :cap].cpu().numpy(), parent[:, :beams], token[:, :beams], lengths)
        st = status_tensor()
        length = t32(lengths)
        orpo.orpo_beam_history(h[:, :cap], t32(parent)[:, :beams], t32(token)[:, :beams], length, st)
        assert int(st.item()) == 0
        assert np.array_equal(h[:, :cap].cpu().numpy(), want)
        assert bool((h[:, cap:] == -7).all()) and bool((flat[:off] == -7).all()) and torch.equal(length, t32(lengths))


def test_cycles_and_many_children():
    h = torch.arange(8, dtype=torch.int32, device=dev()).view(8, 1).repeat(1, 2000)
    st = status_tensor()
    orpo.orpo_beam_history(h, t32([[1, 2, 3, 0, 7, 7, 7, 7]]), t32([[0] * 8]), t32([1999]), st)
    assert h[:, 0].tolist() == h[:, 1998].tolist() == [1, 2, 3, 0, 7, 7, 7, 7] and bool((h[:, 1999] == 0).all())


def test_wrong_entries_are_left_as_they_are():
    first = torch.arange(40, dtype=torch.int32, device=dev()).view(10, 4)
    h = first.clone()
    st = status_tensor()
    orpo.orpo_beam_history(h, t32([[1, 0], [2, 0], [-1, 0], [1, 0], [1, 0]]), t32([[50, 51]] * 5), t32([3, 3, 3, 4, -1]), st)
    assert int(st.item()) == PARENT
    assert torch.equal(h[2:], first[2:])
    assert h[0].tolist() == [4, 5, 6, 50] and h[1].tolist() == [0, 1, 2, 51]


def test_long_histories():
    """More columns than one grid of CTAs has threads for."""
    cap = 9_000_001
    h = torch.stack((torch.arange(cap, dtype=torch.int32, device=dev()), torch.zeros(cap, dtype=torch.int32, device=dev())))
    st = status_tensor()
    orpo.orpo_beam_history(h, t32([[1, 0]]), t32([[5, 6]]), t32([cap - 1]), st)
    assert int(st.item()) == 0 and bool((h[0, :-1] == 0).all()) and h[:, -1].tolist() == [5, 6]
    assert torch.equal(h[1, :-1], torch.arange(cap - 1, dtype=torch.int32, device=dev()))
