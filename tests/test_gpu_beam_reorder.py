"""orpo_beam_reorder against the oracle: moved bytes are equal bytes, and nothing else changes."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu

PARENT = orpo.STATUS_BITS["parent"]


def state_of(shape, dtype=torch.uint8, offset=0, seed=0):
    """Random bytes of the given shape that start `offset` elements into an allocation."""
    size = torch.empty((), dtype=dtype).element_size()
    n = int(np.prod(shape))
    g = torch.Generator("cuda").manual_seed(seed)
    raw = torch.randint(0, 256, ((n + offset + 4) * size,), generator=g, device=dev(), dtype=torch.uint8)
    return raw, raw.view(dtype)[offset:offset + n].view(shape)


def check(shape, parent, length, dtype=torch.uint8, offset=0, status=0, bad=()):
    raw, state = state_of(shape, dtype, offset)
    before_raw, before = raw.cpu().numpy(), state.view(torch.uint8).view(*shape[:4], -1).cpu().numpy()
    p = torch.as_tensor(parent, dtype=torch.int32, device=dev())
    ln = None if length is None else torch.as_tensor(length, dtype=torch.int32, device=dev())
    st = status_tensor()
    orpo.orpo_beam_reorder(state, p, ln, st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    pp = np.array(parent)
    ll = np.full(len(pp), shape[3]) if length is None else np.array(length)
    for b in bad:
        pp[b], ll[b] = np.arange(pp.shape[1]), 0
    ref = oracle.beam_reorder(before, pp, ll)
    assert np.array_equal(state.view(torch.uint8).view(*shape[:4], -1).cpu().numpy(), ref)
    size = state.element_size()
    after = raw.cpu().numpy()
    lo, hi = offset * size, offset * size + before.size
    assert np.array_equal(after[:lo], before_raw[:lo]) and np.array_equal(after[hi:], before_raw[hi:])


@pytest.mark.parametrize("beams", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 64])
def test_beam_counts(beams):
    rng = np.random.default_rng(beams)
    for parent in (rng.integers(0, beams, (3, beams)), np.stack([rng.permutation(beams) for _ in range(3)]),
                   np.stack([np.roll(np.arange(beams), 1), np.arange(beams), np.zeros(beams, dtype=int)])):
        check((2, 3 * beams, 2, 19, 48), parent, [19, 7, 12])


@pytest.mark.parametrize("unit", [1, 2, 3, 4, 6, 8, 12, 16, 24, 33, 64, 72, 128, 136, 512])
@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
def test_unit_sizes_and_alignment(unit, offset):
    check((2, 8, 3, 21, unit), [[1, 2, 3, 0], [0, 0, 2, 1]], [21, 10], offset=offset)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16, torch.int8, torch.float64])
def test_types(dtype):
    check((3, 10, 2, 33, 20), [[4, 3, 2, 1, 0], [2, 2, 2, 2, 2]], [33, 32], dtype=dtype)


@pytest.mark.parametrize("length", [None, [0, 0], [1, 0], [1, 300], [300, 299]])
def test_lengths(length):
    check((2, 6, 2, 300, 32), [[2, 0, 1], [1, 1, 0]], length)


def test_one_position_and_long_ones():
    check((1, 2, 1, 1, 8), [[1, 0]], None)
    check((1, 4, 1, 20000, 64), [[3, 3, 0, 1]], [19999])
    check((300, 2, 1, 5, 16), [[1, 0]], [4])
    check((1, 2 * 700, 5, 3, 16), np.tile([[1, 0]], (700, 1)), None)


@pytest.mark.parametrize("parent,length", [([[1, 4, 0, 2], [3, 2, 1, 0]], [9, 9]), ([[1, -1, 0, 2], [3, 2, 1, 0]], [9, 9]),
                                           ([[1, 0, 0, 2], [3, 2, 1, 0]], [10, 9]), ([[1, 0, 0, 2], [3, 2, 1, 0]], [-1, 9])])
def test_bad_entries_are_reported_and_left_alone(parent, length):
    check((2, 8, 2, 9, 16), parent, length, status=PARENT, bad=[0])


def test_parents_as_columns_of_a_wider_selection():
    _, state = state_of((2, 6, 2, 11, 32))
    before = state.cpu().numpy()
    wide = torch.tensor([[1, 2, 0, 9, 9, 9], [0, 0, 1, 9, 9, 9]], dtype=torch.int32, device=dev())
    st = status_tensor()
    orpo.orpo_beam_reorder(state, wide[:, :3], None, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert np.array_equal(state.cpu().numpy(), oracle.beam_reorder(before, wide[:, :3].cpu().numpy()))


def test_refusals():
    st = status_tensor()
    p = torch.zeros((2, 2), dtype=torch.int32, device=dev())
    _, state = state_of((1, 4, 2, 8, 16))
    for bad in (state.transpose(2, 3), state[0], state[:, :3]):
        with pytest.raises(ValueError):
            orpo.orpo_beam_reorder(bad, p, None, st)
    with pytest.raises(ValueError):
        orpo.orpo_beam_reorder(state, p.long(), None, st)
    with pytest.raises(ValueError):
        orpo.orpo_beam_reorder(state, p.T.contiguous().T, None, st)
    with pytest.raises(ValueError):
        orpo.orpo_beam_reorder(state, p, torch.zeros(3, dtype=torch.int32, device=dev()), st)


def test_offsets_past_32_bits():
    """A state of 8.6 GB whose beams lie 2.1 GB apart, compared on the device."""
    _, state = state_of((1, 4, 1, (1 << 20) + 3, 2048), seed=3)
    rows = torch.tensor([0, 1, 1 << 19, (1 << 20) - 1, (1 << 20) + 1], device=dev())
    last = state[0, :, 0, -1].clone()
    want = state[0, :, 0][:, rows][[1, 3, 2, 0]].clone()
    sums = state.view(4, -1)[[1, 3, 2, 0], :-2048].sum(1, dtype=torch.int64)
    st = status_tensor()
    orpo.orpo_beam_reorder(state, torch.tensor([[1, 3, 2, 0]], dtype=torch.int32, device=dev()),
                           torch.tensor([(1 << 20) + 2], dtype=torch.int32, device=dev()), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(state[0, :, 0][:, rows], want) and torch.equal(state[0, :, 0, -1], last)
    assert torch.equal(state.view(4, -1)[:, :-2048].sum(1, dtype=torch.int64), sums)
