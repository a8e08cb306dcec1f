"""Generates responses by beam search on a quantised head and scores them with the training forward.

The body is a stand-in that needs no checkpoint: hidden state t is a decayed sum of the embeddings of the
tokens so far, kept per beam, so it has to follow its beam's parent like a key/value cache does.  The
beam score of a finished response is then the sum of the per-token log-probabilities that
orpo_head_fwd_q gives for it: both read the same quantised weights (penalties change what is scored, so the two differ
where there are any).  --paged keeps the hidden rows in pages that the beams share.

    python examples/beam_decode.py [--steps 24] [--beams 4] [--paged] [--repetition 1.2] [--no-repeat 3]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import orpo_preference_loss_gb300 as orpo  # noqa: E402
import workloads  # noqa: E402

DECAY = 0.5


def hidden(state):
    return (state / state.norm(dim=-1, keepdim=True).clamp_min(1e-6) * state.shape[-1] ** 0.5).bfloat16()


PAGE = 4  # positions per page


def generate(batch, beams, steps, d=256, V=4096, bits=4, group=64, softcap=30.0, seed=0, paged=False, repetition=1.0, no_repeat=0):
    """Returns (head, quantised weights, responses [batch, beams, steps], their hidden rows)."""
    dev = torch.device("cuda")
    w = workloads.make("tiny", seed=seed, d=d, V=V)
    wq, scales, biases = workloads.quantize_affine(w.W, bits, group)
    bf16 = lambda a: torch.from_numpy(a.view("int16")).to(dev).view(torch.bfloat16)  # noqa: E731
    weights = (torch.from_numpy(wq).to(dev), bf16(scales), bf16(biases))
    g = torch.Generator(dev).manual_seed(seed)
    embedding = torch.randn((V, d), generator=g, device=dev)
    prompt = torch.randint(0, V, (batch,), generator=g, device=dev)

    dec = orpo.BeamDecoder(batch, beams, V, d, bits, group, softcap, eos=1, device=dev, repetition=repetition, no_repeat=no_repeat)
    # per-beam states: the running sum, and what was generated (tokens behind the prompt's, hidden rows) up to length[b]
    running = embedding[prompt].repeat_interleave(beams, 0).view(1, batch * beams, 1, 1, d)
    history = torch.full((batch * beams, steps + 1), 1, dtype=torch.int32, device=dev)
    history[:, 0] = prompt.repeat_interleave(beams)
    length = torch.zeros(batch, dtype=torch.int32, device=dev)
    states, pages, pools = (), None, ()
    if paged:
        columns = steps // PAGE + 1
        pages = orpo.PagedStates(batch, beams, columns, batch * beams * columns, PAGE, status=dec.status, device=dev)
        pool = torch.zeros((1, pages.pages, 1, PAGE, d), dtype=torch.bfloat16, device=dev)
        pools = (pool,)
        pages.advance(length)  # room for the first position
    else:
        rows = torch.zeros((1, batch * beams, 1, steps, d), dtype=torch.bfloat16, device=dev)
        states = (rows,)
    for t in range(steps):
        h = hidden(running.view(-1, d))
        if paged:
            pool[0, pages.table[:, t // PAGE].long(), 0, t % PAGE] = h
        else:
            rows[0, :, 0, t] = h
        length.fill_(t + 1)
        parent, token = dec.step(h, *weights, states=states, length=length, history=history, pages=pages, pools=pools)
        orpo.orpo_beam_reorder(running, parent, None, dec.status)
        running.mul_(DECAY).add_(embedding[token.view(-1).long()].view_as(running))
    if paged:
        at = torch.arange(steps, device=dev)
        rows = pool[0, pages.table[:, at // PAGE].long(), 0, at % PAGE]
    return dec, weights, history[:, 1:].reshape(batch, beams, steps), rows.reshape(batch * beams * steps, d)


def rescore(dec, weights, tokens, rows):
    """Sum of orpo_head_fwd_q's log-probabilities of each response, up to and with its eos."""
    dev = rows.device
    M = rows.shape[0]
    ended = (tokens == dec.eos).int().cumsum(-1)
    counted = ((ended == 0) | ((ended == 1) & (tokens == dec.eos))).to(torch.uint8)
    logp, lse = torch.empty(M, device=dev), torch.empty(M, device=dev)
    ws = torch.empty(orpo.orpo_head_q_workspace_bytes(M, dec.V, dec.d), dtype=torch.uint8, device=dev)
    orpo.orpo_head_fwd_q(rows, *weights, dec.bits, dec.group, tokens.reshape(-1).contiguous(),
                         counted.reshape(-1).contiguous(), dec.softcap, logp, lse, ws, dec.status)
    return logp.view(tokens.shape).sum(-1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--paged", action="store_true")
    ap.add_argument("--repetition", type=float, default=1.0)
    ap.add_argument("--no-repeat", type=int, default=0)
    a = ap.parse_args()
    dec, weights, tokens, rows = generate(a.batch, a.beams, a.steps, paged=a.paged, repetition=a.repetition, no_repeat=a.no_repeat)
    again = rescore(dec, weights, tokens, rows)
    status = int(dec.status.item())
    if status:
        raise SystemExit(orpo.orpo_status_string(status))
    for b in range(a.batch):
        for k in range(a.beams):
            print(f"prompt {b} beam {k}: score {dec.score[b, k].item():9.4f}  training forward {again[b, k].item():9.4f}  "
                  f"tokens {tokens[b, k, :8].tolist()} ...")


if __name__ == "__main__":
    main()
