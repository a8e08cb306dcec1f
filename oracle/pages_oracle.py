"""Oracle of what a decode step does after the logits: their adjustment, the token histories, states in shared pages.

Written from the definitions alone, one token, row and page at a time; shares no code with the library.
"""

from __future__ import annotations

import collections
import math

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def _f32_range(y: float) -> float:
    """What of y fp32's range leaves (values are not rounded)."""
    return math.copysign(math.inf, y) if abs(y) > F32_MAX * (1 + 2.0 ** -25) else y


def logits_adjust(logits, beams, history=None, length=None, prompt=None, repetition=1.0, presence=0.0, frequency=0.0, no_repeat=0,
                  bias_token=None, bias_value=None, masks=None, mask_row=None):
    """(adjusted logits in float64, elementwise bound of an fp32 evaluation's error).

    Each step's result carries one fp32 rounding, at most 2^-24 of its magnitude; so do the penalty itself and each partial
    sum of a token's biases.  repetition, presence, frequency and the biases are the fp32 values that a call passes."""
    x = np.array(logits, dtype=np.float64)
    bound = np.zeros_like(x)
    rows, V = x.shape
    rep, pres, freq = (float(np.float32(p)) for p in (repetition, presence, frequency))
    for r in range(rows):
        b = r // beams
        n = 0 if length is None else int(length[b])
        h = [] if history is None else [int(t) for t in history[r][:n]]
        start = 0 if prompt is None else int(prompt[b])
        count, seen, banned, biases = {}, set(), set(), {}
        for i, t in enumerate(h):
            if 0 <= t < V:
                seen.add(t)
                if i >= start:
                    count[t] = count.get(t, 0) + 1
        if no_repeat and len(h) >= no_repeat:
            end = h[len(h) - (no_repeat - 1):]
            if all(0 <= t < V for t in end):
                for i in range(len(h) - no_repeat + 1):
                    if h[i:i + no_repeat - 1] == end:
                        banned.add(h[i + no_repeat - 1])
        if bias_token is not None:
            tokens, values = (bias_token, bias_value) if np.ndim(bias_token) == 1 else (bias_token[b], bias_value[b])
            for t, v in zip(tokens, values):
                if 0 <= t < V:
                    biases.setdefault(int(t), []).append(float(v))
        for t in seen | set(biases):
            y, err = x[r, t], 0.0
            if t in seen and rep != 1.0:
                y = _f32_range(y / rep if y > 0 else y * rep)
                err += abs(y)
            if count.get(t):
                p = pres + freq * count[t]
                y = _f32_range(y - p)
                err += abs(p) + abs(y)
            if t in biases:
                total = 0.0
                for v in biases[t]:
                    total = _f32_range(total + v)
                    err += abs(total)
                y = _f32_range(y + total)
                err += abs(y)
            x[r, t] = y
            # each rounding is made on a value that carries the ones before it: second order, far below this factor
            bound[r, t] = err * 2.0 ** -24 * (1 + 2.0 ** -16) if math.isfinite(err) else 0.0
        for t in banned:
            if 0 <= t < V:
                x[r, t], bound[r, t] = -math.inf, 0.0
        if masks is not None and mask_row[r] >= 0:
            words = np.array([int(w) & 0xffffffff for w in masks[mask_row[r]]], dtype=np.int64)
            v = np.arange(V)
            masked = (words[v // 32] >> (v % 32)) % 2 == 0
            x[r, masked], bound[r, masked] = -math.inf, 0.0
    return x, bound


def beam_history(history, parent, token, length):
    """A copy of history [batch * beams, capacity] after the step."""
    new = history.copy()
    batch, beams = parent.shape
    for b in range(batch):
        n = int(length[b])
        for k in range(beams):
            new[b * beams + k, :n] = history[b * beams + parent[b, k], :n]
            new[b * beams + k, n] = token[b, k]
    return new


def holders(table, pages):
    """How many entries of table hold each page."""
    refs = np.zeros(pages, dtype=np.int32)
    for e in table.ravel():
        if 0 <= e < pages:
            refs[e] += 1
    return refs


def pages_advance(table, refs, page, parent, length, more, most):
    """(table, refs, moves, full) after a step, taken one row, column and page at a time."""
    table, refs = table.copy(), refs.copy()
    batch = len(length)
    beams = table.shape[0] // batch
    if parent is not None:
        old = table.copy()
        for b in range(batch):
            used = -(-int(length[b]) // page)
            for k in range(beams):
                for c in range(used):
                    was, now = old[b * beams + k, c], old[b * beams + parent[b, k], c]
                    table[b * beams + k, c] = now
                    if now >= 0:
                        refs[now] += 1
                    if was >= 0:
                        refs[was] -= 1
    free = collections.deque(p for p in range(len(refs)) if refs[p] == 0)
    before = table.copy(), refs.copy()
    moves = []
    for r in range(table.shape[0]):
        n = int(length[r // beams])
        m = most if more is None else int(more[r // beams])
        for c in range(n // page, -(-(n + m) // page) if m else 0):
            e = table[r, c]
            if e >= 0 and refs[e] <= 1:
                continue
            if not free:
                return (*before, [], True)
            p = free.popleft()
            if e >= 0:
                refs[e] -= 1
                if c * page < n:
                    moves.append((int(e), p, n - c * page))
            refs[p] = 1
            table[r, c] = p
    return table, refs, moves, False


def pages_copy(pool, moves):
    """A copy of pool [outer, pages, rows, page, unit] after the moves."""
    new = pool.copy()
    for src, dst, n in moves:
        new[:, dst, :, :n] = pool[:, src, :, :n]
    return new


def pages_release(table, refs, ended, beams):
    table, refs = table.copy(), refs.copy()
    for r in range(table.shape[0]):
        if ended is None or ended[r // beams]:
            for e in table[r]:
                if e >= 0:
                    refs[e] -= 1
            table[r] = -1
    return table, refs


def pages_compact(table, refs, page):
    """(table, refs, live, moves) with the pages in use at the lowest numbers."""
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] == 0]
    movers = [p for p in range(live, len(refs)) if refs[p] > 0]
    table, refs = table.copy(), refs.copy()
    for a, b in zip(movers, holes):
        table[table == a] = b
        refs[b], refs[a] = refs[a], 0
    return table, refs, live, [(a, b, page) for a, b in zip(movers, holes)]
