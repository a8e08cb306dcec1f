"""orpo_beam_select against the float64 oracle.  Tolerance of a value: the sum of exp and its log are
off by a few 1e-6 in fp32 (ex2 is good to 2^-22, its argument to 2^-24 of at most ~30), and three
additions round by 2^-24 of their operands; tokens and parents have to be equal wherever the order
does not rest on a difference below that."""

import math

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu

NONFINITE = orpo.STATUS_BITS["nonfinite"]


def run(x, score, beams, n, finished=None, eos=-1, status=0):
    batch = x.shape[0] // beams
    ws = torch.empty(max(16, orpo.orpo_beam_select_workspace_bytes(batch, beams, x.shape[1], n)), dtype=torch.uint8,
                     device=dev())
    ws.fill_(0xA5)
    out = [torch.full((batch, n), 77, dtype=t, device=dev())
           for t in (torch.float32, torch.int32, torch.int32, torch.uint8)]
    st = status_tensor()
    orpo.orpo_beam_select(x, score, finished, eos, beams, *out, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return [o.cpu().numpy() for o in out]


def check(x, score, beams, n, finished=None, eos=-1, status=0):
    got = run(x, score, beams, n, finished, eos, status)
    fin = None if finished is None else finished.cpu().numpy()
    rs, rp, rt, rf, gap = oracle.beam_select(x.double().cpu().numpy(), score.double().cpu().numpy(), fin, eos, beams, n)
    finite = np.isfinite(rs)
    assert np.array_equal(finite, np.isfinite(got[0])) and np.all(got[0][~finite] == -np.inf)
    big = 64 + np.nanmax(np.abs(np.where(np.isfinite(rs), rs, 0)), initial=0)
    tol = 4e-6 + 2.0 ** -22 * big
    assert np.all(np.abs(got[0][finite] - rs[finite]) <= tol)
    for b in range(rs.shape[0]):
        if gap[b] > 2 * tol or gap[b] == 0:
            for g, r in zip(got[1:], (rp, rt, rf)):
                assert np.array_equal(g[b], r[b]), (b, g[b], r[b], gap[b])
    assert np.mean(gap > 2 * tol) > 0.5 or np.any(gap == 0)
    return got


def logits(rows, V, seed, std=2.5, dtype=torch.float32, pitch=0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn((rows, V + pitch), generator=g, device=dev()) * std).to(dtype)[:, :V]
    return x, -10 * torch.rand(rows, generator=g, device=dev())


@pytest.mark.parametrize("V", [1, 2, 3, 31, 64, 255, 1000, 1023, 1025, 4096, 8191, 8193, 16385, 50257, 131072])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabulary_sizes(V, dtype):
    for beams, n in ((1, 1), (4, 8), (3, 3)):
        n = min(n, V)
        x, score = logits(2 * beams, V, V, dtype=dtype)
        check(x, score, beams, n)


@pytest.mark.parametrize("beams,n", [(1, 64), (2, 2), (5, 10), (8, 16), (16, 32), (33, 33), (64, 64), (64, 1), (3, 61)])
@pytest.mark.parametrize("batch", [1, 3])
def test_beams_and_candidates(beams, n, batch):
    x, score = logits(batch * beams, 9001, beams * n + batch)
    check(x, score, beams, n)


@pytest.mark.parametrize("pitch", [1, 3, 4, 8, 13])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_row_pitches_and_alignment(pitch, dtype):
    x, score = logits(8, 20003, pitch, dtype=dtype, pitch=pitch)
    check(x, score, 4, 6)
    x, score = logits(8, 20003, pitch, dtype=dtype, pitch=pitch)
    check(x[:, 1:], score, 4, 6)  # rows that start one element off


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n", [(5000, 16), (40000, 64), (9, 9)])
def test_equal_logits_go_to_the_lowest_token(V, n, dtype):
    g = torch.Generator("cuda").manual_seed(V)
    coarse = torch.randint(0, 4, (6, V), generator=g, device=dev()).to(dtype)
    check(coarse, -torch.arange(6, device=dev(), dtype=torch.float32), 3, n)
    flat = torch.full((6, V), -3.0, dtype=dtype, device=dev())  # every logit equal
    got = check(flat, torch.tensor([0.0, -1.0, -2.0] * 2, device=dev()), 3, n)
    assert got[2][0].tolist() == list(range(n)) and set(got[1].ravel()) == {0}


def test_equal_beams_go_to_the_lower_beam():
    x, _ = logits(1, 3000, 1)
    x = x.expand(8, -1).contiguous()
    got = check(x, torch.zeros(8, device=dev()), 4, 8)
    assert got[1].tolist() == [[0, 1, 2, 3, 0, 1, 2, 3]] * 2
    # the first step of a search: only beam 0 may propose
    score = torch.tensor([0.0] + [-math.inf] * 3, device=dev()).repeat(2)
    got = check(x, score, 4, 8)
    assert np.all(got[1] == 0)
    # scores so low that the logits are lost in them: still each beam's own order
    got = run(x, torch.tensor([0.0, -1e9, -1e9, -1e9] * 2, device=dev()), 4, 4)
    assert np.all(got[1] == 0)


@pytest.mark.parametrize("order", ["ascending", "descending", "spike"])
@pytest.mark.parametrize("n", [1, 16, 64])
def test_orders_that_crowd_the_best_together(order, n):
    V = 33000
    x = torch.linspace(-8, 8, V, device=dev())[None].repeat(4, 1)
    if order == "descending":
        x = x.flip(1).contiguous()
    if order == "spike":
        x = torch.zeros((4, V), device=dev())
        x[:, 12345:12345 + 80] = torch.arange(80, device=dev()) * 0.125
    check(x, torch.tensor([0.0, -0.3, -0.6, -0.9], device=dev()), 2, n)


@pytest.mark.parametrize("value", [-math.inf, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("n", [4, 40])
def test_masks(value, n):
    """Masked tokens, as -inf or the type's lowest value; rows with fewer live tokens than n, and with none."""
    x, score = logits(12, 20000, 7)
    g = torch.Generator("cuda").manual_seed(3)
    x[:, torch.rand(20000, generator=g, device=dev()) < 0.9] = value
    x[1] = value
    x[5, 3:] = value
    x[8:, 10:] = value
    if value == -math.inf:
        check(x, score, 4, n)
    else:  # a row of lowest values has a finite lse: its tokens are equally likely, log(V) is lost in rounding
        got = run(x, score, 4, n)
        keep = [0, 2, 3]
        one, _ = x[keep].contiguous(), None
        alone = run(one, score[keep].contiguous(), 3, min(n, 30))
        assert np.all(np.isfinite(alone[0])) and not np.any(np.isnan(got[0]))
        assert np.all(np.diff(got[0], axis=1) <= 0)
        assert got[0][0, 0] >= score[1].item() - 1e-5  # row 1: score + 0


def test_bf16_lowest_value_as_mask():
    x, score = logits(4, 5000, 11, dtype=torch.bfloat16)
    x[:, 100:] = torch.finfo(torch.bfloat16).min
    check(x, score, 2, 8)


def test_nan_and_inf_are_reported_and_never_selected():
    x, score = logits(8, 6000, 5)
    x[2, 77] = math.nan
    got = check(x, score, 4, 8, status=NONFINITE)
    assert 77 not in got[2][0][got[1][0] == 2]
    x, score = logits(8, 6000, 5)
    x[5, 4] = math.inf
    got = check(x, score, 4, 8, status=NONFINITE)
    assert 1 not in got[1][1]
    x, score = logits(8, 6000, 5)
    score[6] = math.nan
    got = check(x, score, 4, 8, status=NONFINITE)
    assert 2 not in got[1][1]
    x[:, :] = math.nan
    got = check(x, torch.zeros(8, device=dev()), 4, 8, status=NONFINITE)


@pytest.mark.parametrize("n", [4, 9])
def test_finished_beams(n):
    x, score = logits(12, 7001, 13)
    x[1] = math.nan  # a finished beam's logits are not read
    fin = torch.zeros(12, dtype=torch.uint8, device=dev())
    fin[1] = 1
    fin[4:8] = 3  # an entry whose beams are all finished
    score[1] = -0.01
    got = check(x, score, 4, n, finished=fin, eos=5)
    assert got[2][0][0] == 5 and got[3][0][0] == 1
    assert np.all(got[2][1] == 5) and np.all(got[3][1] == 1)
    x[:, 5] = 50.0  # every live beam ends
    x[1, 5] = math.nan
    got = check(x, score, 4, 4, finished=fin, eos=5)
    assert np.all(got[3][0] == 1)


def test_outputs_may_replace_score_and_finished():
    x, score = logits(15, 30001, 17)
    fin = torch.zeros(15, dtype=torch.bool, device=dev())
    fin[7] = True
    ref = run(x, score, 5, 5, finished=fin, eos=9)
    ws = torch.empty(orpo.orpo_beam_select_workspace_bytes(3, 5, 30001, 5), dtype=torch.uint8, device=dev())
    parent, token = (torch.empty((3, 5), dtype=torch.int32, device=dev()) for _ in range(2))
    st, s, f = status_tensor(), score.view(3, 5).clone(), fin.view(3, 5).clone()
    orpo.orpo_beam_select(x, s, f, 9, 5, s, parent, token, f, ws, st)
    for a, b in zip((s, parent, token, f.to(torch.uint8)), ref):
        assert np.array_equal(a.cpu().numpy(), b)


def test_workspace_contents_and_neighbours_do_not_matter():
    """Repeated calls on one dirty workspace, on another stream, give the same bits; the workspace's end holds."""
    x, score = logits(24, 70001, 19)
    ref = run(x, score, 4, 8)
    need = orpo.orpo_beam_select_workspace_bytes(6, 4, 70001, 8)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=dev())
    out = [torch.empty((6, 8), dtype=t, device=dev()) for t in (torch.float32, torch.int32, torch.int32, torch.uint8)]
    st = status_tensor()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        orpo.orpo_beam_select(x, score, None, -1, 4, *out, ws[:need], st, stream=side)
    side.synchronize()
    assert int(st.item()) == 0 and torch.all(ws[need:] == 0xFF)
    for a, b in zip(out, ref):
        assert np.array_equal(a.cpu().numpy(), b)


def test_offsets_past_32_bits():
    """Rows 2^30 + 8 elements apart: the third starts past 2^31 elements."""
    V, pitch = 100_000, (1 << 30) + 8
    flat = torch.empty(2 * pitch + V, device=dev())
    x = torch.as_strided(flat, (3, V), (pitch, 1))
    src, score = logits(3, V, 23)
    x.copy_(src)
    got, ref = run(x, score, 3, 12), run(src, score, 3, 12)
    for a, b in zip(got, ref):
        assert np.array_equal(a, b)


def test_a_vocabulary_of_many_segments():
    V = (1 << 21) + 77
    x, score = logits(3, V, 29)
    x[:, V - 1] = 20.0
    got = check(x, score, 3, 10)
    assert got[2][0][0] == V - 1
