"""BeamDecoder with penalties, masks, histories and shared pages together: against the same search on dense states, against
the oracle step by step, from CUDA graphs, and through a serving batch's turnover."""

import os
import sys

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
import workloads
from gpu_helpers import dev, status_tensor

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beam_decode  # noqa: E402

pytestmark = pytest.mark.gpu

V, D = 4096, 256


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


@pytest.fixture(scope="module")
def weights():
    w = workloads.make("tiny")
    wq, s, b = workloads.quantize_affine(w.W, 4, 64)
    t16 = lambda a: torch.from_numpy(a.view(np.int16)).to(dev()).view(torch.bfloat16)  # noqa: E731
    return torch.from_numpy(wq).to(dev()), t16(s), t16(b)


@pytest.mark.parametrize("batch,beams,kw", [(1, 1, {}), (2, 4, {}), (3, 5, dict(repetition=1.3)), (2, 4, dict(no_repeat=2)), (1, 12, dict(repetition=1.1, no_repeat=3))])
def test_paged_and_dense_states_give_the_same_search(batch, beams, kw):
    steps = 21
    dense = beam_decode.generate(batch, beams, steps, seed=beams, **kw)
    paged = beam_decode.generate(batch, beams, steps, seed=beams, paged=True, **kw)
    assert int(dense[0].status.item()) == 0 and int(paged[0].status.item()) == 0
    assert torch.equal(dense[2], paged[2]) and torch.equal(dense[3], paged[3]) and torch.equal(dense[0].score, paged[0].score)
    if kw.get("no_repeat"):
        for seq in paged[2].view(-1, steps).tolist():
            seq = seq[:seq.index(1)] if 1 in seq else seq
            n = kw["no_repeat"]
            grams = [tuple(seq[i:i + n]) for i in range(len(seq) - n + 1)]
            assert len(grams) == len(set(grams))


def test_steps_against_the_oracle(weights):
    """Every part of a step on the outputs of the one before, each compared with the oracle's."""
    batch, beams, page, steps, cap = 2, 5, 3, 7, 32
    rng = np.random.default_rng(3)
    dec = orpo.BeamDecoder(batch, beams, V, D, softcap=30.0, device=dev(), repetition=1.2, presence=0.3, frequency=0.1, no_repeat=2)
    pages = orpo.PagedStates(batch, beams, 12, 100, page, most=cap, status=dec.status, device=dev())
    pools = (torch.zeros((2, 100, 2, page, 8), dtype=torch.bfloat16, device=dev()), torch.zeros((1, 100, 1, page, 5), dtype=torch.uint8, device=dev()))
    prompt = np.array([7, 4], dtype=np.int32)
    hist = rng.integers(0, 40, (batch * beams, cap)).astype(np.int32)
    history, length = t32(hist), t32(prompt)
    masks = rng.integers(-2**31, 2**31, (3, V // 32)).astype(np.int32)
    bias = (rng.integers(0, V, (batch, 9)).astype(np.int32), rng.standard_normal((batch, 9)).astype(np.float32))
    # prompts: beam 0's pages, then everyone's
    pages.admit(torch.zeros_like(length), length, cap)
    pages.advance(length, parent=t32(np.zeros((batch, beams))), pools=pools)
    table, refs, _, _ = oracle.pages_advance(np.full((batch, 12), -1), np.zeros(100, dtype=np.int32), page, None, [0, 0], prompt, cap)
    full = np.full((batch * beams, 12), -1)
    full[::beams] = table
    table, refs, _, _ = oracle.pages_advance(full, refs, page, np.zeros((batch, beams), dtype=int), prompt, None, 1)
    data = [p.clone() for p in pools]
    follow = {}  # what each beam's positions hold
    for step in range(steps):
        n = length.cpu().numpy()
        # every beam writes something of its own at its newest position
        for r in range(batch * beams):
            for t in range(n[r // beams]) if step == 0 else [n[r // beams] - 1]:
                for i, p in enumerate(pools):
                    p[:, int(pages.table[r, t // page]), :, t % page] = (17 * r + 3 * t + i) % 100 if step else (5 * (r // beams) + t) % 100
                follow[r, t] = (17 * r + 3 * t) % 100 if step else (5 * (r // beams) + t) % 100
        h = torch.randn((batch * beams, D), generator=torch.Generator("cuda").manual_seed(step), device=dev()).bfloat16()
        row = rng.integers(-1, 3, batch * beams).astype(np.int32)
        score = dec.score.clone()
        raw = torch.empty_like(dec.logits)
        orpo.orpo_head_logits_q(h, *weights, 4, 64, 30.0, raw, dec.status)
        parent, token = dec.step(h, *weights, length=length, history=history, prompt=t32(prompt), bias_token=t32(bias[0]),
                                 bias_value=torch.from_numpy(bias[1]).to(dev()), masks=t32(masks), mask_row=t32(row), pages=pages, pools=pools)
        assert int(dec.status.item()) == 0
        want, bound = oracle.logits_adjust(raw.double().cpu().numpy(), beams, hist, n, prompt, 1.2, 0.3, 0.1, 2, *bias, masks, row)
        got = dec.logits.double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            assert np.all((got == want) | (np.abs(got - want) <= bound))
        _, rp, rt, _, gap = oracle.beam_select(got, score.view(-1).cpu().numpy(), None, -1, beams, beams)
        assert np.all(gap > 1e-5)
        assert np.array_equal(parent.cpu().numpy(), rp) and np.array_equal(token.cpu().numpy(), rt)
        hist = oracle.beam_history(hist, rp, rt, n)
        assert np.array_equal(history.cpu().numpy(), hist)
        table, refs, _, _ = oracle.pages_advance(table, refs, page, rp, n, None, 1)
        assert np.array_equal(pages.table.cpu().numpy(), table) and np.array_equal(pages.refs.cpu().numpy(), refs)
        follow = {(b * beams + k, t): follow[b * beams + int(rp[b, k]), t] for b in range(batch) for k in range(beams) for t in range(n[b])}
        for (r, t), x in follow.items():
            assert bool((pools[0][:, table[r, t // page], :, t % page] == x).all()), (step, r, t)
        length += 1
    del data
    # an entry ends, what is left is packed, and nothing of it changes
    before = {(r, t): pools[1][:, table[r, t // page], :, t % page].clone() for r in range(beams, 2 * beams) for t in range(n[1])}
    pages.release(torch.tensor([1, 0], dtype=torch.uint8, device=dev()))
    pages.compact(pools)
    assert int(dec.status.item()) == 0
    table = pages.table.cpu().numpy()
    assert (table[:beams] == -1).all() and table.max() < int(pages.live.item()) == int((pages.refs > 0).sum())
    for (r, t), x in before.items():
        assert torch.equal(pools[1][:, table[r, t // page], :, t % page], x)


def test_two_captured_decoders_that_share_a_workspace_and_status(weights):
    """The whole step out of CUDA graphs, replayed in turns, gives what it gives eagerly."""
    batch, beams, page, cap = 2, 4, 4, 40

    def make():
        dec = orpo.BeamDecoder(batch, beams, V, D, device=dev(), eos=1, repetition=1.2, no_repeat=3)
        pages = orpo.PagedStates(batch, beams, 11, 120, page, status=dec.status, device=dev())
        s = dict(dec=dec, pages=pages, pool=torch.zeros((3, 120, 2, page, 16), dtype=torch.bfloat16, device=dev()),
                 history=torch.zeros((batch * beams, cap), dtype=torch.int32, device=dev()), length=t32([1, 1]), h=torch.zeros((batch * beams, D), dtype=torch.bfloat16, device=dev()))
        pages.advance(torch.zeros_like(s["length"]))
        return s

    def step(s):
        s["dec"].step(s["h"], *weights, length=s["length"], history=s["history"], pages=s["pages"], pools=(s["pool"],))
        s["length"].add_(1)

    def go(states, run):
        out = []
        for i in range(12):
            for j, s in enumerate(states):
                s["h"].copy_(torch.randn((batch * beams, D), generator=torch.Generator("cuda").manual_seed(10 * i + j), device=dev()))
                at = s["length"].view(-1, 1).repeat(1, beams).view(-1).long() - 1
                s["pool"][:, s["pages"].table.gather(1, (at // page)[:, None])[:, 0].long(), :, at % page] = s["h"][:, None, None, :16]
                run(j)
        for s in states:
            assert int(s["dec"].status.item()) == 0
            out += [s["dec"].score.clone(), s["history"].clone(), s["pages"].table.clone(), s["pages"].refs.clone(), s["pool"].clone()]
        return out

    eager = [make(), make()]
    want = go(eager, lambda j: step(eager[j]))
    again = [make(), make()]
    again[1]["pages"].workspace = again[0]["pages"].workspace
    first = [{k: v.clone() for k, v in (("score", s["dec"].score), ("history", s["history"]), ("length", s["length"]), ("table", s["pages"].table), ("refs", s["pages"].refs))} for s in again]
    graphs = []
    for s in again:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    for s, f in zip(again, first):  # a capture runs nothing
        assert torch.equal(s["pages"].table, f["table"]) and torch.equal(s["length"], f["length"])
    for a, b in zip(go(again, lambda j: graphs[j].replay()), want):
        assert torch.equal(a, b)


def test_on_a_stream_of_its_own(weights):
    """Everything on a side stream while the current one is busy."""
    batch, beams = 3, 4
    out = []
    for side in (None, torch.cuda.Stream()):
        dec = orpo.BeamDecoder(batch, beams, V, D, device=dev(), repetition=1.5)
        pages = orpo.PagedStates(batch, beams, 9, 60, 4, most=8, status=dec.status, device=dev())
        pool = torch.zeros((2, 60, 1, 4, 8), device=dev())
        history = torch.arange(batch * beams * 20, dtype=torch.int32, device=dev()).view(batch * beams, 20) % V
        length = t32([3, 7, 8])
        h = torch.randn((batch * beams, D), generator=torch.Generator("cuda").manual_seed(1), device=dev()).bfloat16()
        pages.advance(torch.zeros_like(length), more=length, most=8)
        torch.cuda.synchronize()
        if side is not None:
            torch.cuda._sleep(20_000_000)
        dec.step(h, *weights, length=length, history=history, pages=pages, pools=(pool,), stream=side)
        if side is not None:
            side.synchronize()
        out.append([t.clone() for t in (dec.score, dec.token, history, pages.table, pages.refs)])
        torch.cuda.synchronize()
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_what_a_step_needs_is_asked_for(weights):
    dec = orpo.BeamDecoder(1, 2, V, D, device=dev(), repetition=1.5)
    h = torch.zeros((2, D), dtype=torch.bfloat16, device=dev())
    history = torch.zeros((2, 8), dtype=torch.int32, device=dev())
    with pytest.raises(ValueError, match="history"):
        dec.step(h, *weights)
    with pytest.raises(ValueError, match="length"):
        dec.step(h, *weights, history=history)
    with pytest.raises(ValueError, match="beams"):
        dec.step(h, *weights, history=history, length=t32([1]), pages=orpo.PagedStates(1, 3, 4, 10, 4, device=dev()))
    pages = orpo.PagedStates(1, 2, 4, 10, 4, device=dev())
    with pytest.raises(ValueError, match="pool"):
        pages.compact((torch.zeros((1, 9, 1, 4, 8), device=dev()),))
    with pytest.raises(ValueError, match="pool"):
        pages.advance(t32([0]), pools=(torch.zeros((10, 4, 8), device=dev()),))
    with pytest.raises(ValueError, match="ended"):
        pages.release(torch.zeros(2, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError, match="range"):
        orpo.PagedStates(1, 2, 4, 0, 4, device=dev())
    with pytest.raises(orpo.OrpoError):  # more positions at once than the workspace is for
        pages.advance(t32([0]), most=10_000)


def test_arguments_of_the_wrong_kind_are_refused():
    st, x = status_tensor(), torch.zeros((4, 64), device=dev())
    h = torch.zeros((4, 8), dtype=torch.int32, device=dev())
    two = t32([1, 1])
    bad = [dict(history=h.long(), length=two), dict(history=h, length=two.long()), dict(history=h), dict(history=h, length=t32([1])),
           dict(history=h[:3], length=two), dict(history=h.t(), length=two), dict(history=h, length=two, prompt=two.float()),
           dict(history=h, length=two.cpu()), dict(bias_token=two), dict(bias_token=two, bias_value=two), dict(bias_token=h[:2], bias_value=x[:2, :7]),
           dict(bias_token=h[:2], bias_value=x[:2, :8]), dict(masks=h), dict(mask_row=t32([0] * 4)), dict(masks=h[:, :2], mask_row=two),
           dict(masks=h[:, :1], mask_row=t32([0] * 4)), dict(masks=h[:, :2].float(), mask_row=t32([0] * 4))]
    for kw in bad:
        with pytest.raises((ValueError, orpo.OrpoError)):
            orpo.orpo_logits_adjust(x, 2, st, repetition=1.5, **kw)
    with pytest.raises(ValueError):
        orpo.orpo_logits_adjust(x, 3, st, h, two, repetition=1.5)
    with pytest.raises(ValueError):
        orpo.orpo_logits_adjust(x.half(), 2, st, h, two, repetition=1.5)
    table, refs = torch.full((4, 3), -1, dtype=torch.int32, device=dev()), torch.zeros(9, dtype=torch.int32, device=dev())
    moves, n, ws = torch.zeros((4, 3), dtype=torch.int32, device=dev()), t32([0]), torch.zeros(4096, dtype=torch.uint8, device=dev())
    ok = dict(table=table, refs=refs, page=4, parent=None, length=two, more=None, most=1, moves=moves, n_moves=n, workspace=ws, status=st)
    orpo.orpo_pages_advance(**ok)
    for kw in (dict(table=table.long()), dict(table=table.t()), dict(refs=refs.long()), dict(parent=t32([[0, 0]])), dict(length=two[:1].expand(2)),
               dict(length=t32([1, 1, 1])), dict(more=t32([1])), dict(moves=moves[:, :2]), dict(moves=moves[:3]), dict(n_moves=two), dict(workspace=ws[:16]),
               dict(workspace=ws.view(torch.int32)), dict(status=st.long()), dict(page=0), dict(refs=refs.cpu())):
        with pytest.raises((ValueError, orpo.OrpoError)):
            orpo.orpo_pages_advance(**{**ok, **kw})
    with pytest.raises(ValueError):
        orpo.orpo_pages_copy(torch.zeros((1, 9, 2, 4), device=dev()), moves, n, st)
    with pytest.raises(ValueError):
        orpo.orpo_pages_copy(torch.zeros((1, 9, 2, 4, 6), device=dev())[..., :3], moves, n, st)
    with pytest.raises(ValueError):
        orpo.orpo_pages_release(table, refs, t32([0, 0]), st)
    with pytest.raises(ValueError):
        orpo.orpo_beam_history(h, t32([[0, 0], [0, 0]]), t32([[0, 0, 0], [0, 0, 0]]), two, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and not bool(x.any())
