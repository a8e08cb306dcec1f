"""The selection's oracle on logits so large that their distance to the maximum is all that counts."""

import math

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("value", [0.0, 1e9, -1e9, -1e30, 3e38, float(np.finfo(np.float32).min)])
def test_a_row_of_one_value_is_uniform(value):
    got = oracle.beam_select(np.full((2, 100), value), [-1.0, -2.0], None, -1, 2, 3)
    assert np.allclose(got[0], -1.0 - math.log(100), rtol=0, atol=1e-12) and got[2].tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("shift", [1e6, -1e12])
def test_a_shift_of_the_row_changes_nothing(shift):
    x = np.arange(50.0)[None] * 0.5
    a, b = (oracle.beam_select(y, [0.0], None, -1, 1, 8)[0] for y in (x, x + shift))
    assert np.allclose(a, b, rtol=0, atol=1e-12)
