"""orpo_beam_select on logits far from zero: masks of any finite value over whole chunks or rows, and rows whose
maximum is large.  Compared with the float64 oracle within the tolerance derived in test_gpu_beam_select.py: logits are
exact inputs, and their distance to the row's maximum is what is rounded."""

import math

import numpy as np
import pytest
import torch

from gpu_helpers import dev
from test_gpu_beam_select import check, logits, run

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FILLS = [-1.55e9, -1.768e9, -1.873e9, -2566914048.0, -1e9, -1e30, -3e38, -65504.0, -1e4]


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("dtype,chunk", [(F32, 8192), (BF16, 16384)])
def test_chunks_masked_by_a_finite_value(fill, dtype, chunk):
    """The first two chunks of a row, the last, all but the last, or none; the rest are ordinary logits."""
    V = 5 * chunk
    x, score = logits(8, V, 3, dtype=dtype)
    x[0, :2 * chunk] = fill
    x[1, 4 * chunk:] = fill
    x[2, :4 * chunk] = fill
    x[4, chunk:] = fill
    x[6, :2 * chunk + 5] = fill
    check(x, score, 4, 6)


@pytest.mark.parametrize("fill", FILLS + [torch.finfo(F32).min, 7.0, 1e9, 3e38])
@pytest.mark.parametrize("V", [100, 20000, 70001])
def test_rows_of_one_value(fill, V):
    """Every token of such a beam has probability 1 / V, however large the value: its score minus log V competes with
    the live beams' continuations."""
    x, score = logits(8, V, 5)
    x[1] = fill
    x[4:] = fill
    got = check(x, score, 4, 8)
    alone = run(x[4:].contiguous(), score[4:].contiguous(), 4, 1)
    best = score[4:].double().max().item() - math.log(V)
    assert abs(alone[0][0, 0] - best) <= 4e-6 + 2.0 ** -22 * 84
    assert np.all(np.isfinite(got[0]))


def test_rows_of_the_lowest_bf16_value():
    x, score = logits(8, 40000, 7, dtype=BF16)
    x[1] = torch.finfo(BF16).min
    x[6, 3:] = torch.finfo(BF16).min
    check(x, score, 4, 8)


@pytest.mark.parametrize("shift", [1e3, -1e4, 1e4, 1e5, -1e5])
@pytest.mark.parametrize("V", [1000, 50257])
def test_rows_far_from_zero(shift, V):
    x, score = logits(12, V, 9)
    x += shift
    check(x, score, 3, 5)


def test_one_live_token_among_lowest_values():
    """All but a few tokens at a mask's value: the live ones first, each with its log-probability."""
    x, score = logits(6, 30000, 11)
    keep = x[:, [5, 17, 29000]].clone()
    x[:] = torch.finfo(F32).min
    x[:, [5, 17, 29000]] = keep
    got = check(x, torch.zeros(6, device=dev()), 1, 2)
    assert set(got[2].ravel()) <= {5, 17, 29000}
