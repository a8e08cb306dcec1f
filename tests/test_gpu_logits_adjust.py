"""orpo_logits_adjust against the oracle: every step alone and together, where each can go wrong."""

import math

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu

PARENT, MASK = orpo.STATUS_BITS["parent"], orpo.STATUS_BITS["mask"]
NP = {torch.float32: np.float32}


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def case(batch, beams, V, cap, dtype=torch.float32, pad=0, seed=0, masks=0, n_bias=0, spread=1.0, shared=False):
    """Random inputs; `spread` of the vocabulary is what histories are drawn from."""
    rng = np.random.default_rng(seed)
    rows = batch * beams
    x = torch.from_numpy(rng.standard_normal((rows, V + pad)).astype(np.float32) * 3).to(dev()).to(dtype)[:, :V]
    c = dict(x=x, beams=beams, history=rng.integers(0, max(1, int(V * spread)), (rows, cap)).astype(np.int32),
             length=rng.integers(0, cap + 1, batch).astype(np.int32), prompt=rng.integers(0, cap + 1, batch).astype(np.int32))
    c["length"][-1] = cap
    if n_bias:
        shape = (n_bias,) if shared else (batch, n_bias)
        c["bias_token"] = rng.integers(-1, V + 1, shape).astype(np.int32)
        c["bias_value"] = (rng.standard_normal(shape) * 4).astype(np.float32)
    if masks:
        c["masks"] = rng.integers(-2**31, 2**31, (masks, -(-V // 32))).astype(np.int32)
        c["masks"][0] = 0
        c["masks"][-1] = -1
        c["mask_row"] = rng.integers(-1, masks, rows).astype(np.int32)
        c["mask_row"][0] = 0
    return c


def check(c, repetition=1.0, presence=0.0, frequency=0.0, no_repeat=0, use_prompt=True, want_status=0):
    x = c["x"]
    first = x.double().cpu().numpy()
    whole = torch.as_strided(x, (x.shape[0], x.stride(0)), (x.stride(0), 1)).clone() if x.shape[0] > 1 else None
    prompt = c["prompt"] if use_prompt else None
    more = dict(bias_token=c.get("bias_token"), bias_value=c.get("bias_value"), masks=c.get("masks"), mask_row=c.get("mask_row"))
    want, bound = oracle.logits_adjust(first, c["beams"], c["history"], c["length"], prompt, repetition, presence, frequency, no_repeat,
                                       **more)
    st = status_tensor()
    put = {k: None if v is None else torch.from_numpy(v).to(dev()) for k, v in more.items()}
    orpo.orpo_logits_adjust(x, c["beams"], st, t32(c["history"]), t32(c["length"]), None if prompt is None else t32(prompt), repetition,
                            presence, frequency, no_repeat, **put)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    got = x.double().cpu().numpy()
    if x.dtype is torch.bfloat16:  # the result rounded once: half a unit, 2^-8 of the value
        bound = np.where(bound > 0, bound + 2.0 ** -8 * (np.abs(np.where(np.isfinite(want), want, 0)) + bound), 0)
        big = float(torch.finfo(torch.bfloat16).max) * (1 + 2.0 ** -9)
        want = np.where(np.abs(want) >= big, np.copysign(math.inf, want), want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        assert np.all(same | (np.abs(got - want) <= bound)), np.argwhere(~(same | (np.abs(got - want) <= bound)))[:5]
    if whole is not None:  # what lies between the rows is not touched
        after = torch.as_strided(x, (x.shape[0], x.stride(0)), (x.stride(0), 1))[:-1, x.shape[1]:]
        assert torch.equal(after, whole[:-1, x.shape[1]:])
    return got


# few rows take counters, many (more than two CTAs per SM would hold) a bit per token
SIZES = [(160, 2, 33, 40), (310, 1, 2500, 300), (1, 1, 1, 1), (1, 4, 31, 5), (2, 3, 33, 40), (3, 2, 1000, 300), (1, 1, 8192, 4096), (2, 2, 8193, 1000), (1, 3, 20011, 5000)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("batch,beams,V,cap", SIZES)
@pytest.mark.parametrize("what", ["repetition", "presence", "frequency", "all", "bias", "masks", "ngram", "everything"])
def test_against_the_oracle(batch, beams, V, cap, dtype, what):
    every = what == "everything"
    for pad in (0, 1, 3):
        c = case(batch, beams, V, cap, dtype, pad, seed=pad, masks=5 if what == "masks" or every else 0,
                 n_bias=37 if what == "bias" or every else 0, spread=0.05 if what == "ngram" else 1.0)
        check(c, repetition=1.3 if what in ("repetition", "all") or every else 1.0, presence=0.4 if what in ("presence", "all") or every else 0.0,
              frequency=0.25 if what in ("frequency", "all") or every else 0.0, no_repeat=2 if what == "ngram" or every else 0,
              use_prompt=pad != 1)


@pytest.mark.parametrize("no_repeat,presence,n_bias", [(0, 0.0, 0), (0, 0.4, 5), (2, 0.0, 0), (2, 0.4, 5)])
def test_many_rows_of_long_histories(no_repeat, presence, n_bias):
    """More tokens than a CTA takes at a time, in the form with a bit per token."""
    c = case(1, 310, 700, 3500, seed=no_repeat, masks=3, n_bias=n_bias)
    check(c, 1.2, presence, 0.0, no_repeat)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 32])
def test_n_grams(n):
    """Histories that repeat themselves, with padding inside and lengths around n."""
    rng = np.random.default_rng(n)
    V, cap = 300, 400
    period = rng.integers(0, V, 45)
    h = np.stack([np.resize(period, cap), np.resize(period[:7], cap), np.resize(np.append(period[:6], -1), cap), np.full(cap, 9),
                  rng.integers(0, 3, cap), rng.integers(V, V + 5, cap)]).astype(np.int32)
    h = np.concatenate([h] * 5)
    length = np.repeat([cap, n - 1, n, n + 1, 97], 6).astype(np.int32)
    for times in (1, 12):  # counters, and a bit per token
        x = torch.zeros((30 * times, V), device=dev())
        c = dict(x=x, beams=1, history=np.tile(h, (times, 1)), length=np.tile(length, times), prompt=None)
        got = check(c, no_repeat=n, use_prompt=False)
        assert np.isinf(got[0]).sum() >= 1


def test_history_tokens_outside_the_vocabulary_count_nowhere():
    V = 100
    h = np.array([[-1, 100, 2**31 - 1, -2**31, 5, 99, 0, 101]], dtype=np.int32)
    x = torch.ones((1, V), device=dev())
    got = check(dict(x=x, beams=1, history=h, length=np.array([8]), prompt=np.array([0])), 2.0, 0.5, 0.25)
    assert sorted(np.flatnonzero(got[0] != 1)) == [0, 5, 99]


@pytest.mark.parametrize("prompt", [-5, 0, 3, 8, 100])
def test_the_prompt_counts_for_repetition_alone(prompt):
    h = np.array([[1, 1, 2, 1, 3, 2, 1, 4]], dtype=np.int32)
    check(dict(x=torch.full((1, 10), 3.0, device=dev()), beams=1, history=h, length=np.array([8]), prompt=np.array([max(prompt, 0)])), 2.0, 0.5, 0.25)
    # negative values are as 0
    x = torch.full((1, 10), 3.0, device=dev())
    st = status_tensor()
    orpo.orpo_logits_adjust(x, 1, st, t32(h), t32([8]), t32([prompt]), 2.0, 0.5, 0.25)
    y = torch.full((1, 10), 3.0, device=dev())
    orpo.orpo_logits_adjust(y, 1, st, t32(h), t32([8]), t32([max(prompt, 0)]), 2.0, 0.5, 0.25)
    assert torch.equal(x, y) and int(st.item()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_infinities_nan_and_the_type_s_lowest_value(dtype):
    low = torch.finfo(dtype).min
    vals = [math.inf, -math.inf, math.nan, low, -low, 0.0, -0.0, 1e-42, -1e-42, 2.0]
    V = len(vals)
    masks = np.array([[0], [(1 << V) - 1]], dtype=np.int32)
    for times in (100, 1):
        x = torch.tensor([vals] * 4 * times, device=dev()).to(dtype)
        c = dict(x=x, beams=4 * times, history=np.tile(np.arange(V, dtype=np.int32), (4 * times, 1)), length=np.array([V]), prompt=np.array([0]),
                 masks=masks, mask_row=np.tile(np.array([0, 1, -1, 1], dtype=np.int32), times))
        got = check(c, repetition=1.5, presence=0.25)
    assert np.all(got[0] == -math.inf)  # whatever was there
    assert got[1][0] == math.inf and got[1][1] == -math.inf and math.isnan(got[1][2]) and got[1][3] == -math.inf


def test_bias_lists():
    """The same token twice and more, in the list and in the history; a list for all entries; infinite values; long lists."""
    rng = np.random.default_rng(0)
    for batch, frequency in ((2, 0.1), (2, 0.0), (200, 0.0)):
        c = case(batch, 2, 500, 50, n_bias=300, seed=1)
        c["bias_token"][:, ::3] = 7
        check(c, 1.2, 0.3, frequency)
    c = case(3, 2, 20000, 50, n_bias=64, seed=2, shared=True)
    check(c, 1.2)
    c = case(1, 1, 40, 5, seed=3)
    c["bias_token"], c["bias_value"] = np.array([[3, 4, 3, 5]], dtype=np.int32), np.array([[math.inf, -math.inf, -math.inf, math.nan]], dtype=np.float32)
    got = check(c)
    assert math.isnan(got[0, 3]) and got[0, 4] == -math.inf and math.isnan(got[0, 5])
    c = case(1, 2, 70000, 5, n_bias=4096, seed=4)
    c["bias_token"][0] = rng.permutation(70000)[:4096]
    check(c, 1.1)


def test_order_of_a_bias_s_sum():
    """1e8 + 1 - 1e8 is 0 in fp32 and 1 in another order."""
    x = torch.zeros((1, 9), device=dev())
    st = status_tensor()
    orpo.orpo_logits_adjust(x, 1, st, bias_token=t32([4, 4, 4]), bias_value=torch.tensor([1e8, 1.0, -1e8], device=dev()))
    assert x[0, 4].item() == 0.0 and int(st.item()) == 0


def test_every_word_of_a_mask():
    """One allowed token, and one banned, at each place around word, piece and range borders."""
    V = 8192 + 100
    at = [0, 1, 3, 4, 7, 8, 31, 32, 33, 63, 64, 127, 128, 8159, 8160, 8191, 8192, 8193, V - 2, V - 1]
    for dtype in (torch.float32, torch.bfloat16):
        for pad in (0, 1, 2, 5):
            masks = np.zeros((2 * len(at), -(-V // 32)), dtype=np.uint32)
            for i, v in enumerate(at):
                masks[i, v // 32] = 1 << (v % 32)
                masks[len(at) + i] = 0xffffffff
                masks[len(at) + i, v // 32] ^= np.uint32(1 << (v % 32))
            x = torch.ones((2 * len(at), V + pad), device=dev()).to(dtype)
            st = status_tensor()
            orpo.orpo_logits_adjust(x[:, :V], 1, st, masks=torch.from_numpy(masks.view(np.int32)).to(dev()), mask_row=t32(np.arange(2 * len(at))))
            got = x.float().cpu().numpy()
            want = np.ones_like(got)
            for i, v in enumerate(at):
                want[i, :V] = -math.inf
                want[i, v] = 1
                want[len(at) + i, v] = -math.inf
            assert np.array_equal(got, want) and int(st.item()) == 0


def test_rows_that_a_mask_leaves_nothing_of_and_wrong_mask_numbers():
    V, rows = 100, 5
    masks = torch.zeros((3, 4), dtype=torch.int32, device=dev())
    x = torch.ones((rows, V), device=dev())
    st = status_tensor()
    orpo.orpo_logits_adjust(x, 1, st, masks=masks, mask_row=t32([0, 3, -1, -2, 2]))
    assert int(st.item()) == MASK
    assert torch.all(x[[0, 4]] == -math.inf) and torch.all(x[[1, 2, 3]] == 1)


def test_wrong_lengths_leave_their_entry_as_it_is():
    x = torch.ones((6, 50), device=dev())
    h = t32(np.tile(np.arange(10), (6, 1)))
    st = status_tensor()
    orpo.orpo_logits_adjust(x, 2, st, h, t32([11, 10, -1]), repetition=2.0)
    assert int(st.item()) == PARENT
    assert torch.all(x[[0, 1, 4, 5]] == 1) and torch.all(x[2:4, :10] == 0.5) and torch.all(x[2:4, 10:] == 1)


def test_nothing_behind_length_is_read_and_strided_inputs():
    """Rows of a wider history, bias list and mask table, at odd pitches."""
    rng = np.random.default_rng(5)
    V, rows, cap = 3000, 6, 100
    wide = torch.from_numpy(rng.integers(0, V, (rows, cap + 7)).astype(np.int32)).to(dev())
    x = torch.randn((rows, V), device=dev())
    first = x.double().cpu().numpy()
    length = np.array([0, 1, 100], dtype=np.int32)
    bt = torch.from_numpy(rng.integers(0, V, (3, 9)).astype(np.int32)).to(dev())
    bv = torch.randn((3, 9), device=dev())
    mw = torch.from_numpy(rng.integers(-2**31, 2**31, (4, 101)).astype(np.int32)).to(dev())
    row = np.array([3, -1, 0, 1, 2, 2], dtype=np.int32)
    st = status_tensor()
    orpo.orpo_logits_adjust(x, 2, st, wide[:, 3:cap + 3], t32(length), None, 1.5, 0.0, 0.5, 0, bt[:, 1:6], bv[:, 1:6], mw[:, 2:96], t32(row))
    want, bound = oracle.logits_adjust(first, 2, wide[:, 3:cap + 3].cpu().numpy(), length, None, 1.5, 0.0, 0.5, 0, bt[:, 1:6].cpu().numpy(),
                                       bv[:, 1:6].cpu().numpy(), mw[:, 2:96].cpu().numpy(), row)
    got = x.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        assert np.all((got == want) | (np.abs(got - want) <= bound)) and int(st.item()) == 0


def test_results_repeat_and_counts_are_exact():
    """One token thousands of times among others, counted by many threads at once; bit for bit the same each time."""
    V, cap = 50257, 16384
    rng = np.random.default_rng(9)
    h = rng.integers(0, V, (4, cap)).astype(np.int32)
    h[:, rng.permutation(cap)[:5000]] = 777
    out = []
    for _ in range(3):
        c = case(4, 1, V, cap, seed=3)
        c["history"], c["length"], c["prompt"] = h, np.full(4, cap, dtype=np.int32), np.zeros(4, dtype=np.int32)
        out.append(check(c, 1.1, 0.1, 0.003))
    assert np.array_equal(out[0], out[1]) and np.array_equal(out[0], out[2])


@pytest.mark.parametrize("cap", [40000, 300000])
def test_long_histories(cap):
    c = case(1, 2, 30000, cap, seed=cap)
    c["length"][:] = cap
    check(c, 1.2, 0.1, 0.01, 3)


@pytest.mark.parametrize("frequency", [0.0, 0.25])
@pytest.mark.parametrize("V,cap", [(409600, 500), (409601, 500), (600000, 9000), (1638400, 300), (1638401, 300), (3000000, 200)])
def test_large_vocabularies(V, cap, frequency):
    """On both sides of what fits a CTA's maps of the vocabulary: one, two, three or four of them, for few rows and many."""
    for n_bias, ngram in ((0, 0), (20, 0), (0, 2), (20, 2)):
        for batch in (1, 305 // (2 * -(-V // 32768)) + 1):
            c = case(batch, 2, V, cap, seed=V + n_bias, n_bias=n_bias, spread=0.001 if ngram else 1.0)
            check(c, 1.2, 0.5, frequency, ngram)
    c = case(1, 2, V, cap, seed=V, spread=1e-5)
    check(c, no_repeat=2)


@pytest.mark.parametrize("cap", [8191, 8192])
def test_one_token_all_along(cap):
    """The largest count that 16 bits hold beside their flags, next to counts and flags of its neighbours."""
    for token in (0, 1, 32767, 32768):
        h = np.full((2, cap), token, dtype=np.int32)
        h[1, ::2] = token ^ 1
        c = case(2, 1, 40000, cap, seed=token, n_bias=2)
        c["history"], c["length"], c["prompt"] = h, np.full(2, cap, dtype=np.int32), np.array([0, 5], dtype=np.int32)
        c["bias_token"][:] = [[token ^ 1, 9], [token, token]]
        check(c, 1.5, 0.1, 0.01)


def test_rows_past_2_31_elements():
    """The last rows of 4.4 GB of bf16 logits lie past 2^31 elements."""
    V, rows = 262144, 8300
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device=dev())
    x[-3:] = 2.0
    h = torch.full((rows, 4), -1, dtype=torch.int32, device=dev())
    h[-3:] = t32([[0, 5, 262143, 9]])
    masks = torch.full((1, V // 32), -1, dtype=torch.int32, device=dev())
    masks[0, 3] = 0
    row = torch.full((rows,), -1, dtype=torch.int32, device=dev())
    row[-2:] = 0
    st = status_tensor()
    orpo.orpo_logits_adjust(x, rows, st, h, t32([4]), None, 2.0, masks=masks, mask_row=row)
    want = torch.full((3, V), 2.0, dtype=torch.bfloat16, device=dev())
    want[:, [0, 5, 262143, 9]] = 1.0
    want[1:, 96:128] = -math.inf
    assert int(st.item()) == 0 and torch.equal(x[-3:], want) and not bool(x[:-3].any())


def test_empty_histories_lists_and_batches():
    st, x = status_tensor(), torch.ones((2, 40), device=dev())
    none = torch.empty((2, 0), dtype=torch.int32, device=dev())
    orpo.orpo_logits_adjust(x, 1, st, none, t32([0, 0]), repetition=2.0, no_repeat=2)
    orpo.orpo_logits_adjust(x, 2, st, torch.zeros((2, 5), dtype=torch.int32, device=dev()), t32([0]), repetition=2.0, no_repeat=1)
    orpo.orpo_logits_adjust(x, 1, st, bias_token=none, bias_value=none.float())
    orpo.orpo_logits_adjust(x[:0], 3, st, none[:0], t32([]), repetition=2.0)
    orpo.orpo_logits_adjust(x, 2, st)
    assert bool((x == 1).all()) and int(st.item()) == 0
