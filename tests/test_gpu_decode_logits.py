"""orpo_head_logits_q against the float64 oracle on the dequantised weights, elementwise within the
bound of an fp32-accumulating evaluation."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
import workloads
from gpu_helpers import LOGP_ATOL, dev, f64, status_tensor

pytestmark = pytest.mark.gpu


def make(M, d, V, bits, group, seed=0):
    rng = np.random.default_rng(seed)
    W = workloads.round_bf16((rng.standard_normal((V, d)) * (4.0 / d) ** 0.5).astype(np.float32))
    q = workloads.quantize_affine(W, bits, group)
    h = workloads.round_bf16(rng.standard_normal((M, d)).astype(np.float32))
    return h, q, oracle.dequant_affine(*q, bits, group, d)


def to_dev(h, q):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev())  # noqa: E731
    b = lambda a: t(a.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    return b(h), t(q[0]), b(q[1]), b(q[2])


def run(ht, qt, bits, group, cap, out):
    st = status_tensor()
    logits = torch.full((ht.shape[0], qt[0].shape[0]), float("nan"), dtype=out, device=dev())
    orpo.orpo_head_logits_q(ht, *qt, bits, group, cap, logits, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return logits


def check(logits, h, W, cap):
    got = logits.double().cpu().numpy()
    ref = oracle.head_logits(f64(h), W, cap)
    tol = oracle.logits_error_bound(f64(h), W, cap, logits.dtype == torch.bfloat16)
    assert got.shape == ref.shape and np.all(np.abs(got - ref) <= tol + 1e-30), np.max(np.abs(got - ref) / (tol + 1e-30))


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 24, 33, 64, 65, 130])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_row_counts(M, bits, group):
    h, q, W = make(M, 512, 1031, bits, group, seed=M)
    ht, *qt = to_dev(h, q)
    check(run(ht, qt, bits, group, 0.0, torch.float32), h, W, 0.0)


@pytest.mark.parametrize("d,group", [(8, 8), (40, 8), (64, 64), (72, 24), (96, 32), (136, 8), (160, 160), (256, 16),
                                     (384, 24), (640, 128), (2560, 64), (3840, 32), (4096, 128), (8200, 8), (16384, 64)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [3, 20])
def test_hidden_sizes_and_groups(d, group, bits, M):
    h, q, W = make(M, d, 333, bits, group, seed=d)
    ht, *qt = to_dev(h, q)
    check(run(ht, qt, bits, group, 0.0, torch.float32), h, W, 0.0)


@pytest.mark.parametrize("V", [1, 2, 15, 16, 17, 31, 33, 127, 129, 4096, 50257])
@pytest.mark.parametrize("M", [1, 40])
def test_vocabulary_sizes(V, M):
    h, q, W = make(M, 128, V, 4, 64, seed=V)
    ht, *qt = to_dev(h, q)
    check(run(ht, qt, 4, 64, 0.0, torch.float32), h, W, 0.0)


@pytest.mark.parametrize("cap", [0.5, 30.0, 200.0])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 12, 48])
def test_softcap_and_types(cap, out, M):
    h, q, W = make(M, 320, 700, 4, 32, seed=5)
    ht, *qt = to_dev(h, q)
    check(run(ht, qt, 4, 32, cap, out), h, W, cap)


@pytest.mark.parametrize("M", [3, 33])
def test_row_pitches(M):
    """h as the last positions of hidden states; logits into a wider buffer whose other columns stay."""
    h, q, W = make(M, 256, 1001, 4, 64, seed=9)
    ht, *qt = to_dev(h, q)
    hidden = torch.full((M, 4, 256), float("nan"), dtype=torch.bfloat16, device=dev())
    hidden[:, -1] = ht
    wide = torch.full((M, 1037), 7.0, device=dev())
    st = status_tensor()
    orpo.orpo_head_logits_q(hidden[:, -1], *qt, 4, 64, 0.0, wide[:, :1001], st)
    torch.cuda.synchronize()
    assert torch.all(wide[:, 1001:] == 7.0)
    check(wide[:, :1001], h, W, 0.0)


@pytest.mark.parametrize("offset", [4, 8])
def test_weights_that_start_off_a_16_byte_boundary(offset):
    h, q, W = make(5, 256, 300, 4, 64, seed=2)
    ht, *qt = to_dev(h, q)
    flat = torch.empty(qt[0].numel() + 16, dtype=torch.uint8, device=dev())
    wq = flat[offset:offset + qt[0].numel()].view(qt[0].shape)
    wq.copy_(qt[0])
    a = run(ht, (wq, *qt[1:]), 4, 64, 0.0, torch.float32)
    check(a, h, W, 0.0)


@pytest.mark.parametrize("M", [6, 40])
def test_infinities_and_nan_stay_in_their_row(M):
    h, q, W = make(M, 256, 515, 4, 64, seed=3)
    ht, *qt = to_dev(h, q)
    clean = run(ht, qt, 4, 64, 0.0, torch.float32)
    ht[1, 17] = float("nan")
    ht[4, 200] = float("inf")
    got = run(ht, qt, 4, 64, 0.0, torch.float32)
    keep = [m for m in range(M) if m not in (1, 4)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.all(torch.isnan(got[1])) and not torch.any(torch.isfinite(got[4]))


@pytest.mark.parametrize("M", [2, 33])
@pytest.mark.parametrize("bits", [4, 8])
def test_results_repeat_and_do_not_depend_on_other_rows(M, bits):
    h, q, W = make(M, 768, 5003, bits, 128, seed=4)
    ht, *qt = to_dev(h, q)
    a, b = (run(ht, qt, bits, 128, 30.0, torch.float32) for _ in range(2))
    assert torch.equal(a, b)
    ht[0] = 1e3
    assert torch.equal(run(ht, qt, bits, 128, 30.0, torch.float32)[1:], a[1:])


@pytest.mark.parametrize("bits,group,cap", [(4, 64, 30.0), (8, 32, 0.0)])
def test_agrees_with_the_training_forward(bits, group, cap):
    """log_softmax of these logits at the target is the logp orpo_head_fwd_q gives for it."""
    w = workloads.make("tiny")
    q = workloads.quantize_affine(w.W, bits, group)
    ht, *qt = to_dev(w.h, q)
    logits = run(ht, qt, bits, group, cap, torch.float32)
    ws = torch.empty(orpo.orpo_head_q_workspace_bytes(w.M, w.V, w.d), dtype=torch.uint8, device=dev())
    tg = torch.from_numpy(w.targets).to(dev())
    mask = torch.ones(w.M, dtype=torch.uint8, device=dev())
    logp, lse, st = torch.empty(w.M, device=dev()), torch.empty(w.M, device=dev()), status_tensor()
    orpo.orpo_head_fwd_q(ht, *qt, bits, group, tg, mask, cap, logp, lse, ws, st)
    ours = torch.log_softmax(logits.double(), 1).gather(1, tg.long()[:, None])[:, 0]
    assert torch.max(torch.abs(ours - logp)) < LOGP_ATOL


def test_offsets_past_32_bits():
    """4.6 GB of weights and logits rows 2^30 elements apart; a sample of rows against the oracle."""
    V, d, group, M = 1_100_003, 8192, 128, 3
    g = torch.Generator("cuda").manual_seed(1)
    wq = torch.randint(0, 256, (V, d // 2), generator=g, device=dev(), dtype=torch.uint8)
    sc = (torch.rand((V, d // group), generator=g, device=dev()) * 0.01).bfloat16()
    bi = (sc.float() * -7.5).bfloat16()
    h = torch.randn((M, d), generator=g, device=dev()).bfloat16()
    flat = torch.empty(2 * (1 << 30) + V, device=dev())
    logits = torch.as_strided(flat, (M, V), (1 << 30, 1))
    st = status_tensor()
    orpo.orpo_head_logits_q(h, wq, sc, bi, 4, group, 0.0, logits, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    rows = torch.tensor([0, 1, 524287, 524288, 524289, 1_048_575, 1_048_576, V - 2, V - 1], device=dev())
    bits16 = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    W = oracle.dequant_affine(wq[rows].cpu().numpy(), bits16(sc[rows]), bits16(bi[rows]), 4, group, d)
    ref = oracle.head_logits(f64(bits16(h)), W)
    tol = oracle.logits_error_bound(f64(bits16(h)), W, 0.0, False)
    assert np.all(np.abs(logits[:, rows].double().cpu().numpy() - ref) <= tol)
