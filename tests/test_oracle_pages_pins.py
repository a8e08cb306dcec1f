"""Hand-worked cases of the oracle of the logits' adjustment, the histories and the shared pages."""

import math

import numpy as np

import oracle

I = lambda *a: np.array(a, dtype=np.int32)  # noqa: E731, E741


def test_penalties_by_hand():
    x = np.array([[4.0, -4.0, 4.0, -4.0, 0.0, 4.0]])
    h = I([0, 1, 1, 2, 3, 9, -1])
    y, bound = oracle.logits_adjust(x, 1, h, [7], [1], 2.0, 0.5, 0.25)
    # token 0 stands in the prompt alone; 1 twice; 2 and 3 once; 9 and -1 are no tokens
    assert y.tolist() == [[2.0, -8.0 - 1.0, 2.0 - 0.75, -8.0 - 0.75, 0.0, 4.0]]
    assert bound[0, 4] == bound[0, 5] == 0.0 and np.all(bound[0, :4] > 0)


def test_n_grams_by_hand():
    x = np.zeros((1, 8))
    ban = lambda h, n: [v for v in range(8) if oracle.logits_adjust(x, 1, I(h), [len(h)], None, no_repeat=n)[0][0, v] < 0]  # noqa: E731
    assert ban([1, 2, 3, 1, 2], 3) == [3]
    assert ban([1, 2, 3, 1, 2, 4, 1, 2], 3) == [3, 4]
    assert ban([1, 2, 3], 1) == [1, 2, 3]
    assert ban([1, 2, 3], 2) == [] and ban([3, 3], 2) == [3] and ban([3, 3, 3], 3) == [3]
    assert ban([1, 2], 3) == [] and ban([], 1) == []
    assert ban([-1, 3, 4, -1], 2) == []  # padding is no n-gram
    assert ban([9, 3, 4, 9], 2) == []


def test_biases_and_masks_by_hand():
    x = np.array([[1.0, 2.0, 3.0, math.inf]])
    y, _ = oracle.logits_adjust(x, 1, bias_token=I(1, 2, 1, 7, -3), bias_value=np.float32([1, 2, 4, 8, 16]), masks=I([0b0110]), mask_row=[0])
    assert y.tolist() == [[-math.inf, 7.0, 5.0, -math.inf]]
    y, _ = oracle.logits_adjust(x, 1, masks=I([0b0110]), mask_row=[-1])
    assert np.array_equal(y, x)


def test_overflow_is_fp32_s():
    x = np.array([[-3.4e38, 3.4e38]])
    y, _ = oracle.logits_adjust(x, 1, I([0, 1]), [2], None, 1.5)
    assert y[0, 0] == -math.inf and math.isfinite(y[0, 1])


def test_history_by_hand():
    h = I([1, 2, 9, 9], [3, 4, 8, 8], [5, 6, 7, 7], [0, 0, 0, 0])
    new = oracle.beam_history(h, I([1, 1], [1, 0]), I([10, 11], [12, 13]), [2, 1])
    assert new.tolist() == [[3, 4, 10, 9], [3, 4, 11, 8], [0, 12, 7, 7], [5, 13, 0, 0]]


def test_a_step_of_pages_by_hand():
    # two beams, pages of 4: a full page shared, a page each with two positions of it in use
    table = I([0, 2, -1], [0, 3, -1])
    refs = oracle.holders(table, 6)
    assert refs.tolist() == [2, 0, 1, 1, 0, 0]
    # both follow beam 1: page 2 is let go of and, being the lowest but one free page, page 1 is beam 0's copy
    t, r, moves, full = oracle.pages_advance(table, refs, 4, I([1, 1]), [6], None, 1)
    assert t.tolist() == [[0, 1, -1], [0, 3, -1]] and r.tolist() == [2, 1, 0, 1, 0, 0] and moves == [(3, 1, 2)] and not full
    # a page boundary: new pages, none copied
    t, r, moves, full = oracle.pages_advance(table, refs, 4, None, [8], None, 1)
    assert t.tolist() == [[0, 2, 1], [0, 3, 4]] and moves == [] and not full
    # not enough pages
    t, r, moves, full = oracle.pages_advance(table, refs, 4, None, [4], I(5), 5)
    assert t.tolist() == [[0, 2, 1], [0, 3, 4]]
    t, r, moves, full = oracle.pages_advance(table, oracle.holders(table, 4), 4, None, [8], None, 1)
    assert full and np.array_equal(t, table) and moves == []
    # rewriting a shared full page: beam 0 gets a page of its own, nothing of the old one is kept
    t, r, moves, full = oracle.pages_advance(table, refs, 4, None, [0], None, 4)
    assert t.tolist() == [[1, 2, -1], [0, 3, -1]] and moves == []


def test_release_and_compact_by_hand():
    table = I([5, 2], [5, 3], [0, -1])
    refs = oracle.holders(table, 7)
    t, r = oracle.pages_release(table, refs, [1, 0, 0], 1)
    assert t.tolist() == [[-1, -1], [5, 3], [0, -1]] and r.tolist() == [1, 0, 0, 1, 0, 1, 0]
    t, r, live, moves = oracle.pages_compact(t, r, 4)
    assert live == 3 and moves == [(3, 1, 4), (5, 2, 4)]
    assert t.tolist() == [[-1, -1], [2, 1], [0, -1]] and r.tolist() == [1, 1, 1, 0, 0, 0, 0]
