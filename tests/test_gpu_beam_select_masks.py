"""orpo_beam_select on logits far from zero: masks of any finite value over whole chunks.  Compared with the float64 oracle within the tolerance derived in test_gpu_beam_select.py: logits are
exact inputs, and their distance to the row's maximum is what is rounded."""

import pytest
import torch

from gpu_helpers import dev
from test_gpu_beam_select import check, logits

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


def test_one_live_token_among_lowest_values():
    """All but a few tokens at a mask's value: the live ones first, each with its log-probability."""
    x, score = logits(6, 30000, 11)
    keep = x[:, [5, 17, 29000]].clone()
    x[:] = torch.finfo(F32).min
    x[:, [5, 17, 29000]] = keep
    got = check(x, torch.zeros(6, device=dev()), 1, 2)
    assert set(got[2].ravel()) <= {5, 17, 29000}
