"""Decode calls shared by the bounds-checked-build test and the child process it starts: every kernel and ring form, the
rare paths of the selection, and every form of the reordering.  Each case returns its outputs and the status word."""

import numpy as np
import torch

import orpo_preference_loss_gb300 as orpo

LOGITS = [  # M, d, V, bits, group, h's pitch beyond d, logits' pitch beyond V, bytes the weights and values the scales are off
    (1, 256, 4096, 4, 64, 0, 0, 0, 0), (13, 3840, 5005, 4, 32, 8, 3, 0, 0), (20, 3232, 1111, 4, 32, 0, 0, 0, 0),
    (5, 832, 1000, 4, 64, 0, 0, 0, 1), (2, 1056, 777, 4, 32, 0, 5, 0, 0), (64, 4096, 3000, 4, 128, 0, 0, 0, 0),
    (130, 768, 901, 4, 96, 16, 0, 0, 0), (33, 640, 129, 8, 640, 0, 0, 0, 0), (8, 2048, 4003, 8, 32, 0, 0, 0, 0),
    (3, 5376, 501, 8, 64, 0, 0, 0, 0), (17, 160, 333, 8, 32, 0, 0, 0, 0), (4, 512, 700, 4, 32, 0, 0, 8, 0),
    (9, 136, 333, 4, 8, 0, 1, 0, 0), (3, 72, 250, 8, 24, 0, 0, 8, 0), (1, 32, 1, 4, 32, 0, 0, 0, 0)]
SELECT = [  # batch, beams, V, n, bf16, pitch beyond V, what the logits are
    (2, 4, 4096, 4, False, 0, "random"), (3, 5, 20003, 7, False, 3, "random"), (3, 5, 20003, 7, True, 5, "random"),
    (1, 2, 70001, 64, True, 0, "random"), (2, 3, 33000, 16, False, 0, "sorted"), (2, 3, 33000, 40, True, 1, "equal"),
    (2, 4, 20000, 40, False, 0, "masked"), (2, 4, 40000, 8, True, 0, "lowest"), (1, 64, 3000, 64, False, 0, "random"),
    (2, 2, 600000, 9, False, 1, "random"), (4, 1, 1, 1, True, 0, "random"), (2, 4, 9000, 8, False, 0, "nan")]
REORDER = [  # shape, bytes off
    ((2, 8, 3, 21, 64), 0), ((2, 8, 3, 21, 72), 0), ((2, 8, 3, 21, 36), 4), ((3, 16, 2, 1003, 33), 1),
    ((2, 18, 3, 150, 48), 0), ((2, 18, 3, 150, 24), 8), ((2, 34, 1, 77, 20), 0), ((1, 64, 2, 501, 7), 3), ((2, 12, 2, 9000, 16), 0)]
CASES = [("logits", c) for c in LOGITS] + [("select", c) for c in SELECT] + [("reorder", c) for c in REORDER]


def off(t, by):
    flat = torch.empty(t.numel() + 64, dtype=t.dtype, device=t.device)
    m = flat[by:by + t.numel()].view(t.shape)
    m.copy_(t)
    return m


def run_case(op, c, seed=1):
    dev = torch.device("cuda:0")
    g = torch.Generator("cuda").manual_seed(seed)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    if op == "logits":
        M, d, V, bits, group, hp, lp, wo, so = c
        wq = off(torch.randint(0, 256, (V, d * bits // 8), generator=g, device=dev, dtype=torch.uint8), wo)
        sc = off((torch.rand((V, d // group), generator=g, device=dev) * 0.01).bfloat16(), so)
        bi = off((sc.float() * -7.5).bfloat16(), so)
        h = torch.randn((M, d + hp), generator=g, device=dev).bfloat16()[:, :d]
        wide = torch.zeros((M, V + lp), device=dev)
        orpo.orpo_head_logits_q(h, wq, sc, bi, bits, group, 30.0, wide[:, :V], st)
        out = [wide]
    elif op == "select":
        batch, beams, V, n, bf16, pad, what = c
        x = torch.randn((batch * beams, V + pad), generator=g, device=dev) * 2.5
        if what == "sorted":
            x = x.sort(1).values
        elif what == "equal":
            x[:] = 1.5
        elif what == "masked":
            x[:, 11:] = float("-inf")
            x[1] = float("-inf")
        elif what == "lowest":
            x[:, 5:] = torch.finfo(torch.bfloat16 if bf16 else torch.float32).min
        elif what == "nan":
            x[:, 70] = float("nan")
        x = (x.bfloat16() if bf16 else x)[:, :V]
        out = [torch.empty((batch, n), dtype=t, device=dev) for t in (torch.float32, torch.int32, torch.int32, torch.uint8)]
        ws = torch.empty(orpo.orpo_beam_select_workspace_bytes(batch, beams, V, n), dtype=torch.uint8, device=dev)
        score = -torch.rand(batch * beams, generator=g, device=dev)
        finished = torch.zeros(batch * beams, dtype=torch.uint8, device=dev)
        finished[-1] = beams > 1
        orpo.orpo_beam_select(x, score, finished, V // 2, beams, *out, ws, st)
    else:
        shape, by = c
        rng = np.random.default_rng(seed)
        beams = shape[1] // 2
        state = off(torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8), by)
        parent = torch.from_numpy(rng.integers(0, beams, (2, beams)).astype(np.int32)).to(dev)
        length = torch.tensor([shape[3], shape[3] - 3], dtype=torch.int32, device=dev)
        orpo.orpo_beam_reorder(state, parent, length, st)
        out = [state]
    torch.cuda.synchronize()
    return {**{f"out{i}": t.cpu().numpy() for i, t in enumerate(out)}, "status": np.array([int(st.item())])}
