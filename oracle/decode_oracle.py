"""Float64 oracle of one beam-search step: logits, selection, state reordering.

Written from the definitions alone (plain loops over batch entries and beams); shares no code with the
library.
"""

from __future__ import annotations

import math

import numpy as np


def head_logits(h: np.ndarray, W: np.ndarray, softcap: float = 0.0) -> np.ndarray:
    """[M, V] logits of rows h under weights W (both float64), softcapped when softcap > 0."""
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.asarray(h, dtype=np.float64) @ np.asarray(W, dtype=np.float64).T
        return softcap * np.tanh(z / softcap) if softcap > 0 else z


def logits_error_bound(h: np.ndarray, W: np.ndarray, softcap: float, out_bf16: bool) -> np.ndarray:
    """Elementwise bound of an fp32-accumulating evaluation of head_logits.

    A sum of d exact products in fp32, in any order and with truncating adds, is off by at most
    d * 2^-23 times the sum of the products' magnitudes.  The softcap (slope at most 1) adds its own
    evaluation error, at most 2^-21 of the cap, and a bf16 result half a unit in its last place, at
    most 2^-8 of its value.
    """
    mag = np.abs(h) @ np.abs(W).T
    tol = h.shape[1] * 2.0 ** -23 * mag
    if softcap > 0:
        tol = tol + softcap * 2.0 ** -21
    if out_bf16:
        tol = tol + 2.0 ** -8 * (np.abs(head_logits(h, W, softcap)) + tol)
    return tol


def beam_select(logits, score, finished, eos: int, beams: int, n: int):
    """(score, parent, token, finished, gap) of the n best continuations per entry.

    gap[b]: the least difference between values that the order among the first n + 1 proposals of
    different beams rests on (inf if none): where it is large against rounding, an evaluation in fp32
    must give the same parents and tokens."""
    x = np.array(logits, dtype=np.float64)
    x[np.isnan(x)] = -math.inf
    batch = x.shape[0] // beams
    out_s, out_p, out_t, out_f, gaps = [], [], [], [], []
    for b in range(batch):
        props = []  # (value, beam, rank, token, finished)
        for k in range(beams):
            r = b * beams + k
            s = float(score[r])
            if finished is not None and finished[r]:
                for j in range(n):
                    v = s if j == 0 and not math.isnan(s) else -math.inf
                    props.append((v, k, j, eos, True))
                continue
            row = x[r]
            top = row.max()
            # lse = top + log_sum, as two numbers: a mask's value of 1e30 leaves nothing of log_sum in one
            log_sum = math.log(np.sum(np.exp(row - top))) if math.isfinite(top) else 0.0
            order = np.argsort(-row, kind="stable")[:n]
            for j, t in enumerate(order):
                ok = row[t] > -math.inf and math.isfinite(top) and not math.isnan(s)
                props.append((s + ((row[t] - top) - log_sum) if ok else -math.inf, k, j, int(t), False))
        props.sort(key=lambda p: (-p[0], p[1], p[2]))
        gap = math.inf
        for p, q in zip(props[:n], props[1:n + 1]):
            if p[1] != q[1] and math.isfinite(p[0]) and math.isfinite(q[0]):
                gap = min(gap, p[0] - q[0])
        gaps.append(gap)
        best = props[:n]
        out_s.append([p[0] for p in best])
        out_p.append([p[1] for p in best])
        out_t.append([p[3] for p in best])
        out_f.append([int(p[4] or p[3] == eos) for p in best])
    return (np.array(out_s), np.array(out_p, dtype=np.int32), np.array(out_t, dtype=np.int32),
            np.array(out_f, dtype=np.uint8), np.array(gaps))


def beam_reorder(state: np.ndarray, parent: np.ndarray, length=None) -> np.ndarray:
    """A reordered copy of state [outer, batch * beams, rows, capacity, unit]."""
    batch, beams = parent.shape
    new = state.copy()
    for b in range(batch):
        used = state.shape[3] if length is None else int(length[b])
        for k in range(beams):
            new[:, b * beams + k, :, :used] = state[:, b * beams + int(parent[b, k]), :, :used]
    return new
