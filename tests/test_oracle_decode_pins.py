"""Pins for the decode oracle: hand-worked selections and reorderings, and the selection against a
flat log-softmax + sort in torch."""

import math

import numpy as np
import pytest
import torch

import oracle


def test_selection_by_hand():
    # two beams, three tokens; equal logits inside a beam go to the lower token
    x = [[0.0, 1.0, 1.0], [2.0, 2.0, -math.inf]]
    lse0, lse1 = math.log(1 + 2 * math.e), math.log(2) + 2
    s, p, t, f, gap = oracle.beam_select(x, [-1.0, -1.5], None, -1, 2, 3)
    # values: beam 0: -1 + 1 - lse0 = -1.862 (tokens 1, 2); beam 1: -1.5 - ln 2 = -2.193 (tokens 0, 1)
    assert p.tolist() == [[0, 0, 1]] and t.tolist() == [[1, 2, 0]] and f.tolist() == [[0, 0, 0]]
    assert np.allclose(s, [[-lse0, -lse0, 0.5 - lse1]])
    assert gap[0] == pytest.approx(-lse0 - 0.5 + lse1)
    # equal values of different beams go to the lower beam
    s, p, t, _, gap = oracle.beam_select([[1.0, 0.0], [1.0, 0.0]], [0.0, 0.0], None, -1, 2, 2)
    assert p.tolist() == [[0, 1]] and t.tolist() == [[0, 0]] and gap[0] == 0.0


def test_finished_masked_and_broken_beams_by_hand():
    nan, ninf = math.nan, -math.inf
    # a finished beam proposes eos at its score, then eos at -inf
    s, p, t, f, _ = oracle.beam_select([[9.0, 9.0], [0.0, 0.0]], [-0.5, -4.0], [1, 0], 1, 2, 2)
    assert p.tolist() == [[0, 1]] and t.tolist() == [[1, 0]] and f.tolist() == [[1, 0]]
    assert s[0, 0] == -0.5 and s[0, 1] == pytest.approx(-4 - math.log(2))
    # a fully masked beam and one with +inf only give -inf; a NaN logit counts as masked
    s, p, t, _, _ = oracle.beam_select([[ninf, ninf], [math.inf, 0.0], [nan, 0.0]], [0.0, 0.0, 0.0], None, -1, 3, 2)
    assert s.tolist() == [[0.0, ninf]] and p.tolist() == [[2, 0]] and t.tolist() == [[1, 0]]
    s, p, _, _, _ = oracle.beam_select([[0.0, 0.0], [0.0, 0.0]], [nan, -1.0], None, -1, 2, 2)
    assert p.tolist() == [[1, 1]]


@pytest.mark.parametrize("beams,n", [(1, 1), (3, 4), (5, 10)])
def test_selection_matches_flat_sort(beams, n):
    g = torch.Generator().manual_seed(beams)
    x = torch.randn((2 * beams, 37), generator=g, dtype=torch.float64)
    score = -torch.rand(2 * beams, generator=g, dtype=torch.float64)
    s, p, t, _, _ = oracle.beam_select(x.numpy(), score.numpy(), None, -1, beams, n)
    flat = (score[:, None] + torch.log_softmax(x, 1)).view(2, -1)
    v, at = flat.sort(1, descending=True)
    assert np.allclose(s, v[:, :n].numpy())
    assert np.array_equal(p, (at // 37)[:, :n].numpy()) and np.array_equal(t, (at % 37)[:, :n].numpy())


def test_reorder_by_hand():
    state = np.arange(2 * 3 * 1 * 2 * 1).reshape(2, 3, 1, 2, 1)
    out = oracle.beam_reorder(state, np.array([[1, 0, 1]]), np.array([1]))
    assert out[0, :, 0, :, 0].tolist() == [[2, 1], [0, 3], [2, 5]]
    assert np.array_equal(oracle.beam_reorder(state, np.array([[0, 1, 2]])), state)


def test_logits_and_their_bound():
    h, W = np.array([[1.0, -2.0]]), np.array([[3.0, 1.0], [0.5, 0.25]])
    assert oracle.head_logits(h, W).tolist() == [[1.0, 0.0]]
    assert oracle.head_logits(h, W, 2.0)[0, 0] == pytest.approx(2 * math.tanh(0.5))
    assert np.allclose(oracle.logits_error_bound(h, W, 0.0, False), [[2 * 2.0 ** -23 * 5, 2 * 2.0 ** -23]])
