"""The three decode operators together: a whole beam search, eager and from a CUDA graph."""

import os
import sys

import numpy as np
import pytest
import torch

import oracle
import orpo_preference_loss_gb300 as orpo
import workloads
from gpu_helpers import dev, f64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beam_decode  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,beams,softcap", [(1, 1, 0.0), (2, 4, 30.0), (3, 5, 30.0)])
def test_scores_are_the_training_forward_s(batch, beams, softcap):
    steps = 20
    dec, weights, tokens, rows = beam_decode.generate(batch, beams, steps, softcap=softcap, seed=beams)
    again = beam_decode.rescore(dec, weights, tokens, rows)
    assert int(dec.status.item()) == 0
    # each of the forward's log-probabilities is within 2e-3 of the exact one
    assert torch.max(torch.abs(again - dec.score)) < steps * 2e-3
    assert torch.all(dec.score[:, :-1] >= dec.score[:, 1:])
    flat = tokens.view(batch, beams, steps).cpu().numpy()
    for b in range(batch):
        assert len({tuple(r) for r in flat[b]}) == beams  # beams hold different responses


def test_steps_match_the_oracle_s_search():
    """Three steps whose hidden rows depend on the token alone, against the float64 oracle."""
    V, d, batch, beams = 4096, 256, 2, 3
    w = workloads.make("tiny")
    wq, s, b = workloads.quantize_affine(w.W, 4, 64)
    W64 = oracle.dequant_affine(wq, s, b, 4, 64, d)
    t16 = lambda a: torch.from_numpy(a.view(np.int16)).to(dev()).view(torch.bfloat16)  # noqa: E731
    weights = (torch.from_numpy(wq).to(dev()), t16(s), t16(b))
    table = workloads.round_bf16(np.random.default_rng(1).standard_normal((V, d)).astype(np.float32))
    table_t = t16(table)
    dec = orpo.BeamDecoder(batch, beams, V, d, device=dev())
    token = torch.tensor([[5] * beams, [900] * beams], dtype=torch.int32, device=dev())
    score, prev = np.array([0.0, -np.inf, -np.inf] * batch), token.cpu().numpy()
    state = torch.arange(batch * beams, dtype=torch.float32, device=dev()).view(1, -1, 1, 1, 1)
    follow = state.cpu().numpy()
    for _ in range(3):
        parent, token = dec.step(table_t[token.view(-1).long()], *weights, states=(state,))
        rs, rp, rt, _, gap = oracle.beam_select(oracle.head_logits(f64(table[prev.ravel()]), W64), score, None, -1, beams,
                                                beams)
        assert np.all(gap > 1e-4)
        assert np.array_equal(parent.cpu().numpy(), rp) and np.array_equal(token.cpu().numpy(), rt)
        assert np.max(np.abs(dec.score.cpu().numpy() - rs)) < 1e-4
        follow = oracle.beam_reorder(follow, rp)
        assert np.array_equal(state.cpu().numpy(), follow)
        score, prev = rs.ravel(), rt
    assert int(dec.status.item()) == 0


def test_a_step_in_a_cuda_graph():
    V, d, batch, beams = 4096, 256, 2, 4
    w = workloads.make("tiny")
    wq, s, b = workloads.quantize_affine(w.W, 4, 64)
    t16 = lambda a: torch.from_numpy(a.view(np.int16)).to(dev()).view(torch.bfloat16)  # noqa: E731
    weights = (torch.from_numpy(wq).to(dev()), t16(s), t16(b))
    h = torch.randn((batch * beams, d), device=dev()).bfloat16()
    cache = torch.randn((4, batch * beams, 2, 64, 32), device=dev()).bfloat16()
    first = cache.clone()
    length = torch.tensor([64, 17], dtype=torch.int32, device=dev())

    def steps(dec, state, replay=None):
        dec.reset()
        out = []
        for i in range(4):
            h.copy_(torch.randn((batch * beams, d), generator=torch.Generator("cuda").manual_seed(i), device=dev()))
            if replay:
                replay()
            else:
                dec.step(h, *weights, states=(state,), length=length)
            out += [dec.parent.clone(), dec.token.clone(), dec.score.clone()]
        return out + [state.clone()]

    dec = orpo.BeamDecoder(batch, beams, V, d, softcap=30.0, eos=1, device=dev())
    eager = steps(dec, cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.step(h, *weights, states=(cache,), length=length)
    cache.copy_(first)
    for a, c in zip(steps(dec, cache, graph.replay), eager):
        assert torch.equal(a, c)


def test_sizes_out_of_range_are_refused():
    with pytest.raises(ValueError):
        orpo.BeamDecoder(1, 65, 4096, 256)
    with pytest.raises(ValueError):
        orpo.BeamDecoder(1, 8, 4, 256)  # fewer tokens than beams
