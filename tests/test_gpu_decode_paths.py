"""The decode operators where their kernels change form or hand things on: rings under load, scales of every
magnitude, group counts that are no multiple of a segment's, workspaces, streams, and calls that follow one
another without a synchronise."""

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
import workloads
from gpu_helpers import dev, f64, status_tensor

pytestmark = pytest.mark.gpu


def random_head(V, d, bits, group, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    top = 2 ** bits - 1
    wq = torch.randint(0, 256, (V, d * bits // 8), generator=g, device=dev(), dtype=torch.uint8)
    sc = (torch.rand((V, d // group), generator=g, device=dev()) * (4.0 / d) ** 0.5 / top).bfloat16()
    return wq, sc, (sc.float() * (-top / 2)).bfloat16()


def rows_of(M, d, seed):
    return torch.randn((M, d), generator=torch.Generator("cuda").manual_seed(seed), device=dev()).bfloat16()


def bits16(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def run(h, q, bits, group, cap=0.0, **kw):
    st = status_tensor()
    out = torch.full((h.shape[0], q[0].shape[0]), float("nan"), device=dev())
    orpo.orpo_head_logits_q(h, *q, bits, group, cap, out, st, **kw)
    return out, st


def check(out, h, q, bits, group, rows=slice(None)):
    W = oracle.dequant_affine(q[0][rows].cpu().numpy(), bits16(q[1][rows]), bits16(q[2][rows]), bits, group, h.shape[1])
    h64 = f64(bits16(h))
    err = np.abs(out[:, rows].double().cpu().numpy() - oracle.head_logits(h64, W))
    assert np.all(err <= oracle.logits_error_bound(h64, W, 0.0, False) + 1e-30)


@pytest.mark.parametrize("M,d,V,bits,group", [(1, 2560, 40000, 4, 64), (13, 3840, 20000, 4, 32), (16, 512, 5000, 4, 32),
                                              (20, 16384, 333, 4, 64), (20, 4096, 20000, 4, 64), (64, 4096, 20000, 4, 128),
                                              (8, 2048, 32000, 8, 32), (40, 4096, 5000, 8, 64), (130, 1024, 9001, 8, 128)])
def test_repeated_calls_give_the_same_bits(M, d, V, bits, group):
    """Every ring wraps many times, with the memory system busy; all calls agree with the first, and that one with
    the oracle on a sample of the vocabulary."""
    q, h = random_head(V, d, bits, group, seed=d), rows_of(M, d, seed=M)
    first, st = run(h, q, bits, group)
    check(first, h, q, bits, group, torch.from_numpy(np.unique(np.linspace(0, V - 1, 97).astype(np.int64))))
    again = [run(h, q, bits, group)[0] for _ in range(6)]
    wrong = torch.zeros((), dtype=torch.int64, device=dev())
    for _ in range(12):
        for out in again:
            out.fill_(float("nan"))
            orpo.orpo_head_logits_q(h, *q, bits, group, 0.0, out, st)
        for out in again:
            wrong += (out != first).sum()
    assert int(wrong.item()) == 0 and int(st.item()) == 0


@pytest.mark.parametrize("d,group", [(832, 64), (768, 384), (1280, 256), (640, 640), (1536, 512), (3264, 64), (3328, 128),
                                     (3360, 32), (5120, 32), (960, 96)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 16, 24])
def test_group_counts(d, group, bits, M):
    q, h = random_head(301, d, bits, group, seed=d + group), rows_of(M, d, seed=M)
    check(run(h, q, bits, group)[0], h, q, bits, group)


@pytest.mark.parametrize("offset", [2, 4, 8])
def test_scales_off_a_16_byte_boundary(offset):
    q, h = random_head(700, 1024, 4, 64, seed=1), rows_of(5, 1024, seed=2)
    moved = []
    for t in q[1:]:
        flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=dev())
        m = flat[offset // 2:offset // 2 + t.numel()].view(t.shape)
        m.copy_(t)
        moved.append(m)
    a, b = run(h, q, 4, 64)[0], run(h, (q[0], *moved), 4, 64)[0]
    check(b, h, q, 4, 64)
    assert torch.equal(a, b)


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32), (4, 32)])
def test_scales_of_every_magnitude(bits, group, M):
    """Blocks of rows whose scales are all small, some large, zero, subnormal, infinite or NaN."""
    V, d = 512, 512
    wq, sc, bi = random_head(V, d, bits, group, seed=bits)
    sc[40:50] *= 1000          # a block of 32 with some large ones
    sc[64:96] = 0.75           # all large
    sc[100] = 2.0 ** -5        # the least that is not small
    sc[101, 0] = 2.0 ** -5 * (1 - 2.0 ** -8)  # the largest that is
    sc[130:140] = 0.0
    sc[160:192] = 2.0 ** -130  # subnormal, with biases that leave the products visible
    bi[160:192] = 2.0 ** -126
    sc[200:210] *= -1
    sc[256:288] = -0.5
    bi[300] = 1e30
    bad = [330, 390, 391]
    sc[330, 1], sc[390, 0], bi[391, 3] = float("inf"), float("nan"), float("inf")
    q, h = (wq, sc, bi), rows_of(M, d, seed=4)
    out, st = run(h, q, bits, group)
    good = torch.tensor([v for v in range(V) if v not in bad])
    check(out, h, q, bits, group, good)
    assert not torch.any(torch.isfinite(out[:, bad])) and int(st.item()) == 0


@pytest.mark.parametrize("M,V", [(17, 100), (33, 128), (64, 129), (20, 19457), (64, 38913), (20, 2 * 152 * 128)])
@pytest.mark.parametrize("d", [384, 1568])
def test_pairs_of_tiles(M, V, d):
    """Odd tile counts, single tiles, and vocabularies that just begin another round of tiles."""
    q, h = random_head(V, d, 4, 32, seed=V), rows_of(M, d, seed=M)
    check(run(h, q, 4, 32)[0], h, q, 4, 32)


@pytest.mark.parametrize("M,d,bits", [(17, 1600, 4), (3, 5376, 4), (3, 5376, 8), (70, 960, 8)])
def test_workspace_contents_and_size(M, d, bits):
    q, h = random_head(1000, d, bits, 64, seed=3), rows_of(M, d, seed=5)
    need = orpo.orpo_head_logits_q_workspace_bytes(M, d, bits)
    assert need > 0
    a, _ = run(h, q, bits, 64)
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b, _ = run(h, q, bits, 64, workspace=ws)
    c, st = run(h, q, bits, 64, workspace=ws.clone(), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c) and torch.all(ws[need:] == 0xff) and int(st.item()) == 0
    with pytest.raises(orpo.OrpoError):
        run(h, q, bits, 64, workspace=ws[:need - 1])


@pytest.mark.parametrize("M,d", [(4, 512), (20, 512), (20, 2048), (4, 5376)])
def test_calls_follow_one_another_without_a_synchronise(M, d):
    """Each step's inputs are written right before it and its outputs read right after it, on one stream: what is set
    up early must wait for both."""
    V, beams, batch = 20000, M // 2, 2
    q = random_head(V, d, 4, 64, seed=7)
    hs = [rows_of(M, d, seed=i) for i in range(4)]
    heads = [random_head(V, d, 4, 64, seed=20 + i) for i in range(2)]
    ws = torch.empty(orpo.orpo_beam_select_workspace_bytes(batch, beams, V, beams), dtype=torch.uint8, device=dev())
    new = lambda dt: torch.empty((batch, beams), dtype=dt, device=dev())  # noqa: E731

    def step(h, head, sync):
        wait = torch.cuda.synchronize if sync else lambda: None
        x = torch.empty_like(h)
        st = status_tensor()
        score, out = torch.zeros((batch, beams), device=dev()), (new(torch.float32), new(torch.int32), new(torch.int32), new(torch.uint8))
        logits = torch.full((M, V), float("nan"), device=dev())
        state = torch.arange(2 * M * 3 * 50 * 33, device=dev(), dtype=torch.int16).view(2, M, 3, 50, 33)
        wait()
        for dst, src in zip(q, head):
            dst.copy_(src)
        x.copy_(h)
        wait()
        orpo.orpo_head_logits_q(x, *q, 4, 64, 30.0, logits, st)
        wait()
        orpo.orpo_beam_select(logits, score, None, -1, beams, *out, ws, st)
        wait()
        orpo.orpo_beam_reorder(state, out[1], None, st)
        wait()
        orpo.orpo_beam_reorder(state, out[1], None, st)
        wait()
        return logits.clone(), out[0], out[1], out[2], state.clone(), st

    cases = [(h, head) for h in hs for head in heads]
    want = [step(h, head, True) for h, head in cases]
    for _ in range(10):
        for (h, head), w in zip(cases, want):
            got = step(h, head, False)
            assert all(torch.equal(x, y) for x, y in zip(got, w))


def test_concurrent_streams():
    """Calls on several streams share the card (and its tensor memory) and do not disturb one another."""
    q = random_head(9000, 1024, 4, 64, seed=9)
    hs = [rows_of(m, 1024, seed=m) for m in (1, 6, 20, 50)]
    want = [run(h, q, 4, 64)[0] for h in hs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in hs]
    outs, sts = [], []
    for _ in range(8):
        for h, s in zip(hs, streams):
            with torch.cuda.stream(s):
                out, st = run(h, q, 4, 64)
                outs.append(out)
                sts.append(st)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % len(hs)]) and int(sts[i].item()) == 0


@pytest.mark.parametrize("unit,beams", [(33, 4), (66, 9), (33, 64), (7, 3), (36, 12), (72, 9), (20, 17), (16, 9)])
def test_reorder_of_long_runs_of_any_unit(unit, beams):
    """Runs of many windows, from sources and to destinations at every byte of 16."""
    rng = np.random.default_rng(unit)
    shape = (2, 2 * beams, 3, 1003, unit)
    state = torch.randint(0, 256, shape, generator=torch.Generator("cuda").manual_seed(unit), device=dev(), dtype=torch.uint8)
    before = state.cpu().numpy()
    parent, length = rng.integers(0, beams, (2, beams)), np.array([1003, 777])
    parent[1, 0] = 0
    st = status_tensor()
    orpo.orpo_beam_reorder(state, torch.from_numpy(parent.astype(np.int32)).to(dev()),
                           torch.from_numpy(length.astype(np.int32)).to(dev()), st)
    assert np.array_equal(state.cpu().numpy(), oracle.beam_reorder(before, parent, length)) and int(st.item()) == 0


def test_select_of_a_chain_of_finished_rows():
    """Every beam finished: nothing of the logits is read, and the step still waits for what came before it."""
    batch, beams, V = 3, 4, 50000
    st = status_tensor()
    ws = torch.empty(orpo.orpo_beam_select_workspace_bytes(batch, beams, V, beams), dtype=torch.uint8, device=dev())
    logits = torch.full((batch * beams, V), float("nan"), device=dev())
    out = [torch.empty((batch, beams), dtype=d, device=dev()) for d in (torch.float32, torch.int32, torch.int32, torch.uint8)]
    for i in range(20):
        score = torch.arange(batch * beams, device=dev(), dtype=torch.float32).view(batch, beams) * -1.0 - i
        finished = torch.ones((batch, beams), dtype=torch.uint8, device=dev())
        orpo.orpo_beam_select(logits, score, finished, 7, beams, *out, ws, st)
        assert torch.equal(out[0], score) and torch.all(out[2] == 7) and torch.all(out[3] == 1)
    assert int(st.item()) == 0


@pytest.mark.parametrize("tail", [1, 7, 8, 100, 255, 256, 257, 500, 1000, 1800, 1816, 2040, 2047])
@pytest.mark.parametrize("n", [1, 5, 64])
@pytest.mark.parametrize("dtype,chunk", [(torch.float32, 8192), (torch.bfloat16, 16384)])
def test_select_with_a_short_last_chunk(tail, n, dtype, chunk):
    V, g = 2 * chunk + tail, torch.Generator("cuda").manual_seed(tail)
    logits = (torch.randn((2, V), generator=g, device=dev()) * 2.5).to(dtype)
    score, st = torch.zeros((1, 2), device=dev()), status_tensor()
    out = [torch.empty((1, n), dtype=d, device=dev()) for d in (torch.float32, torch.int32, torch.int32, torch.uint8)]
    ws = torch.empty(orpo.orpo_beam_select_workspace_bytes(1, 2, V, n), dtype=torch.uint8, device=dev())
    orpo.orpo_beam_select(logits, score, None, -1, 2, *out, ws, st)
    x = logits.double().cpu().numpy()
    ref = oracle.beam_select(x, np.zeros(2), None, -1, 2, n)
    assert int(st.item()) == 0 and np.max(np.abs(out[0].cpu().numpy() - ref[0])) < 1e-5
    # where values of different beams are closer than their rounding, their order may differ
    if ref[4][0] > 1e-5:
        assert np.array_equal(out[1].cpu().numpy(), ref[1]) and np.array_equal(out[2].cpu().numpy(), ref[2])


@pytest.mark.parametrize("d,group", [(832, 64), (1056, 32), (896, 32), (1152, 128), (160, 32)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [2, 20])
def test_a_row_does_not_see_the_next_row_s_scales(d, group, bits, M):
    """Group counts that end inside a segment of columns: infinities and NaN of every third row stay there."""
    V = 385
    wq, sc, bi = random_head(V, d, bits, group, seed=d)
    sc[1::3], bi[1::3] = float("nan"), float("inf")
    out, st = run(rows_of(M, d, seed=1), (wq, sc, bi), bits, group)
    good = torch.tensor([v for v in range(V) if v % 3 != 1])
    check(out, rows_of(M, d, seed=1), (wq, sc, bi), bits, group, good)
    assert not torch.any(torch.isfinite(out[:, 1::3])) and int(st.item()) == 0
