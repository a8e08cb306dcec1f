"""One step of beam search on the quantised head, operator by operator: inputs, plain forms and sizes.

  logits   orpo_head_logits_q: the logits of a few rows of h under the 4/8-bit affine group-quantised head
  select   orpo_beam_select:   log-softmax, and the n best continuations over beams and vocabulary
  reorder  orpo_beam_reorder:  the beams' states (key/value caches) follow their parents, in place

Head sizes are those of the recipes in workloads/ (tiny, small, e4b, largev, ragged).
"""

import random

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"fp32": F32, "bf16": BF16, "u8": torch.uint8}
NINF = float("-inf")


def listed():
    return [
        # the smallest head: one row, a call whose launch is most of its time
        dict(name="logits tiny 1 row", op="logits", M=1, d=256, V=4096, bits=4, group=64, cap=0.0, out="fp32", steps=1),
        # greedy decoding of one sequence on the e4b head (262k tokens, softcap): the weights are read once
        dict(name="logits e4b 1 row", op="logits", M=1, d=2560, V=262144, bits=4, group=64, cap=30.0, out="fp32", steps=1),
        # eight beams on an 8-bit head
        dict(name="logits small 8 rows 8-bit", op="logits", M=8, d=2048, V=32000, bits=8, group=32, cap=0.0, out="bf16", steps=1),
        # sixteen prompts of four beams on the head with the longest rows
        dict(name="logits largev 64 rows", op="logits", M=64, d=4096, V=128256, bits=4, group=128, cap=0.0, out="fp32", steps=1),
        # odd row count and vocabulary; h are the last positions of [M, 5, d] hidden states
        dict(name="logits ragged 13 rows", op="logits", M=13, d=3840, V=50257, bits=4, group=32, cap=30.0, out="bf16", steps=5),
        # one prompt, four beams, small vocabulary: latency
        dict(name="select tiny", op="select", B=1, K=4, V=4096, n=4, x="fp32", pad=0, finished=0, masked=0.0),
        # four prompts, four beams, twice as many candidates as beams (the caller keeps those that go on)
        dict(name="select e4b", op="select", B=4, K=4, V=262144, n=8, x="fp32", pad=0, finished=0, masked=0.0),
        # a large batch with wide beams, 16-bit logits
        dict(name="select largev wide", op="select", B=32, K=8, V=128256, n=16, x="bf16", pad=0, finished=0, masked=0.0),
        # odd sizes, odd row pitch, finished beams, a grammar's mask over 30% of the vocabulary
        dict(name="select odd masked", op="select", B=7, K=5, V=50257, n=5, x="fp32", pad=3, finished=2, masked=0.3),
        # a short cache of one prompt: latency
        dict(name="reorder tiny", op="reorder", N=2, B=1, K=4, R=2, T=128, D=64, x="bf16", longest=100, moved=3, sources=2),
        # the caches of eight layers (keys and values), full to capacity
        dict(name="reorder cache", op="reorder", N=16, B=8, K=4, R=4, T=1024, D=128, x="bf16", longest=1024, moved=3, sources=2),
        # ragged lengths in a longer allocation, positions of 72 bytes
        dict(name="reorder ragged", op="reorder", N=6, B=5, K=6, R=3, T=777, D=36, x="bf16", longest=601, moved=4, sources=3),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["logits", "select", "reorder"])
    if op == "logits":
        while True:
            M, V = _log(rng, 1, 64), _log(rng, 4096, 262144)
            d, bits, group = 32 * _log(rng, 8, 128), rng.choice([4, 4, 8]), rng.choice([32, 64, 128])
            if d % group == 0 and d != 3072 and V != 3072 and V * d * bits <= 262144 * 2560 * 4 and M * V * d <= 64 * 128256 * 4096:
                return dict(op=op, M=M, d=d, V=V, bits=bits, group=group, cap=rng.choice([0.0, 30.0]),
                            out=rng.choice(["fp32", "bf16"]), steps=rng.choice([1, 1, 3]))
    if op == "select":
        while True:
            B, K, V = _log(rng, 1, 32), rng.randint(2, 16), _log(rng, 1000, 262144)
            if B * K * V <= 32 * 8 * 128256 and V != 3072:
                return dict(op=op, B=B, K=K, V=V, n=rng.choice([K, 2 * K]), x=rng.choice(["fp32", "bf16"]),
                            pad=rng.choice([0, 0, 1, 8]), finished=rng.choice([0, 0, 1]), masked=rng.choice([0.0, 0.0, 0.5]))
    while True:
        N, B, K, R = _log(rng, 2, 32), _log(rng, 1, 16), rng.randint(2, 10), rng.randint(1, 8)
        T, D = _log(rng, 64, 4096), rng.choice([32, 64, 80, 128, 256, 36, 33])
        if 2 * N * B * K * R * T * D <= 2 * 16 * 8 * 4 * 4 * 1024 * 128 and 3072 not in (T, D):
            moved = rng.randint(1, K)
            return dict(op=op, N=N, B=B, K=K, R=R, T=T, D=D, x=rng.choice(["bf16", "bf16", "fp32", "u8"]), longest=rng.randint(1 + T // 2, T),
                        moved=moved, sources=rng.randint(1, moved) if moved > 1 else 1)


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _lengths(c):
    """Evenly spread over the upper half of the longest."""
    return [c["longest"] - (c["longest"] // 2) * b // c["B"] for b in range(c["B"])]


def _parents(c, r):
    """Per batch entry: `moved` beams take another beam's state, from `sources` different ones."""
    rows = []
    for _ in range(c["B"]):
        while True:
            p = list(range(c["K"]))
            src = r.sample(p, c["sources"])
            slots = r.sample(range(c["K"]), c["moved"])
            took = [src[i % len(src)] for i in range(len(slots))]
            r.shuffle(took)
            if all(a != b for a, b in zip(slots, took)):
                break
        for a, b in zip(slots, took):
            p[a] = b
        rows.append(p)
    return rows


def prepare(case, seed):
    c, g, dev = case, _gen(seed), "cuda"
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    if c["op"] == "logits":
        M, d, V, group = c["M"], c["d"], c["V"], c["group"]
        top = (1 << c["bits"]) - 1
        wq = torch.empty((V, d * c["bits"] // 8), dtype=torch.uint8, device=dev)
        scales = torch.empty((V, d // group), dtype=BF16, device=dev)
        biases = torch.empty_like(scales)
        for v in range(0, V, 32768):  # W ~ N(0, 4/d), quantised by the range of each group
            w = torch.randn((min(32768, V - v), d // group, group), generator=g, device=dev) * (2.0 / d ** 0.5)
            lo = w.amin(-1)
            s = ((w.amax(-1) - lo) / top).to(BF16)
            b = lo.to(BF16)
            q = ((w - b.float()[..., None]) / s.float()[..., None]).round_().clamp_(0, top).to(torch.uint8).view(-1, d)
            scales[v:v + len(w)], biases[v:v + len(w)] = s, b
            wq[v:v + len(w)] = q if c["bits"] == 8 else q[:, 0::2] | (q[:, 1::2] << 4)
        h = torch.randn((M, c["steps"], d), generator=g, device=dev).to(BF16)[:, -1]
        return dict(c=c, h=h, wq=wq, scales=scales, biases=biases, status=status,
                    logits=torch.empty((M, V), dtype=TYPES[c["out"]], device=dev))
    if c["op"] == "select":
        B, K, V, n = c["B"], c["K"], c["V"], c["n"]
        x = torch.randn((B * K, V + c["pad"]), generator=g, device=dev) * 2.5
        if c["masked"]:
            x[:, torch.rand(V + c["pad"], generator=g, device=dev) < c["masked"]] = NINF
        logits = x.to(TYPES[c["x"]])[:, :V]
        score = -10.0 * torch.rand(B * K, generator=g, device=dev)
        finished = None
        if c["finished"]:
            finished = (torch.rand((B, K), generator=g, device=dev).argsort(1) < c["finished"]).to(torch.uint8).view(-1)
        # a workspace of 16 bytes for each of n + 1 entries of every 1024 logits of a row is always enough
        ws = torch.empty(16 * B * K * (n + 1) * -(-V // 1024) + 4096, dtype=torch.uint8, device=dev)
        out = [torch.empty((B, n), dtype=t, device=dev) for t in (F32, torch.int32, torch.int32, torch.uint8)]
        return dict(c=c, logits=logits, score=score, finished=finished, eos=V // 2, out=out, ws=ws, status=status)
    r = random.Random(seed)
    shape = (c["N"], c["B"] * c["K"], c["R"], c["T"], c["D"])
    if c["x"] == "u8":
        state = torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8)
    else:
        state = torch.randn(shape, generator=g, device=dev).to(TYPES[c["x"]])
    lens = _lengths(c)
    r.shuffle(lens)
    return dict(c=c, state=state, parent=torch.tensor(_parents(c, r), dtype=torch.int32, device=dev),
                length=torch.tensor(lens, dtype=torch.int32, device=dev), status=status)


def run(state):
    op = state["c"]["op"]
    return {"logits": _logits, "select": _select, "reorder": _reorder}[op](state)


def _logits(s):
    c = s["c"]
    if own:
        import orpo_preference_loss_gb300 as orpo
        orpo.orpo_head_logits_q(s["h"], s["wq"], s["scales"], s["biases"], c["bits"], c["group"], c["cap"], s["logits"], s["status"])
        return s["logits"]
    q = s["wq"]
    if c["bits"] == 4:
        q = torch.stack((q & 15, q >> 4), -1)
    q = q.view(c["V"], c["d"] // c["group"], c["group"]).float()
    # the head's weights are bf16 values by definition: bf16(scale q + bias)
    w = (q * s["scales"].float()[..., None] + s["biases"].float()[..., None]).to(BF16).float().view(c["V"], c["d"])
    z = s["h"].float() @ w.T
    if c["cap"] > 0:
        z = c["cap"] * torch.tanh(z / c["cap"])
    return z.to(TYPES[c["out"]])


def _select(s):
    c = s["c"]
    B, K, n = c["B"], c["K"], c["n"]
    if own:
        import orpo_preference_loss_gb300 as orpo
        orpo.orpo_beam_select(s["logits"], s["score"], s["finished"], s["eos"], K, *s["out"], s["ws"], s["status"])
        return s["out"]
    x = s["logits"].float() + 0.0
    x = torch.where(x != x, NINF, x)
    m = x.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(1, keepdim=True))
    best, token = torch.sort(x, dim=1, descending=True, stable=True)
    best, token = best[:, :n], token[:, :n]
    value = s["score"][:, None] + (best - lse)
    value = torch.where((best > NINF) & torch.isfinite(lse) & (value == value), value, NINF)
    over = torch.zeros_like(value, dtype=torch.bool) if s["finished"] is None else (s["finished"] != 0)[:, None].expand(-1, n)
    first = torch.where(torch.arange(n, device=x.device) == 0, s["score"][:, None], NINF)
    value = torch.where(over, first, value).view(B, K * n)
    token = torch.where(over, s["eos"], token).view(B, K * n)
    value, at = torch.sort(value, dim=1, descending=True, stable=True)
    value, at = value[:, :n], at[:, :n]
    parent, token = at // n, token.gather(1, at)
    ended = over[:, 0].view(B, K).gather(1, parent) | (token == s["eos"])
    return [value, parent.to(torch.int32), token.to(torch.int32), ended.to(torch.uint8)]


def _reorder(s):
    c, x = s["c"], s["state"]
    if own:
        import orpo_preference_loss_gb300 as orpo
        orpo.orpo_beam_reorder(x, s["parent"], s["length"], s["status"])
        return x
    v = x.view(c["N"], c["B"], c["K"], c["R"], c["T"], c["D"])
    at = torch.arange(c["B"], device=x.device)[:, None]
    live = torch.arange(c["T"], device=x.device)[None, :] < s["length"][:, None]
    v.copy_(torch.where(live[None, :, None, None, :, None], v[:, at, s["parent"].long()], v))
    return x


def work(case):
    c = case
    if c["op"] == "logits":
        w = c["V"] * c["d"]
        out = c["M"] * c["V"] * (4 if c["out"] == "fp32" else 2)
        return {"bytes": w * c["bits"] / 8 + 4 * w / c["group"] + 2 * c["M"] * c["d"] + out, "flops": 2 * c["M"] * w}
    if c["op"] == "select":
        live = c["B"] * (c["K"] - c["finished"])
        return {"bytes": live * c["V"] * (4 if c["x"] == "fp32" else 2) + 5 * c["B"] * c["K"] + 13 * c["B"] * c["n"], "flops": 4 * live * c["V"]}
    size = {"fp32": 4, "bf16": 2, "u8": 1}[c["x"]]
    return {"bytes": c["N"] * c["R"] * sum(_lengths(c)) * c["D"] * size * (c["moved"] + c["sources"]), "flops": 0}


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "logits":
        h = s["h"].double()
        z = torch.empty((c["M"], c["V"]), dtype=torch.float64, device=h.device)
        for v in range(0, c["V"], 16384):
            rows = slice(v, min(v + 16384, c["V"]))
            q = s["wq"][rows].to(torch.int16)
            full = torch.empty((q.shape[0], c["d"]), dtype=torch.float64, device=h.device)
            if c["bits"] == 4:
                full[:, 0::2], full[:, 1::2] = (q % 16).double(), (q // 16).double()
            else:
                full[:] = q.double()
            scale = s["scales"][rows].double().repeat_interleave(c["group"], 1)
            full.mul_(scale).add_(s["biases"][rows].double().repeat_interleave(c["group"], 1))
            z[:, rows] = h @ full.to(BF16).double().T
        return z if c["cap"] == 0 else c["cap"] * torch.tanh(z / c["cap"])
    if c["op"] == "select":
        B, K, n = c["B"], c["K"], c["n"]
        logp = torch.log_softmax(s["logits"].double(), 1)
        value = (s["score"].double()[:, None] + logp).view(B, K, c["V"])
        rows = []
        for b in range(B):
            parts = []
            for k in range(K):
                if s["finished"] is not None and int(s["finished"][b * K + k]):
                    parts.append(s["score"][b * K + k].double().view(1))
                else:
                    parts.append(value[b, k].topk(n).values)
            rows.append(torch.cat([*parts, torch.full((n,), NINF, dtype=torch.float64, device=value.device)]).topk(n).values)
        return [torch.stack(rows), None, None, None]
    old, new = s["state"].double(), s["state"].double()
    for b, (parents, length) in enumerate(zip(s["parent"].tolist(), s["length"].tolist())):
        for k, p in enumerate(parents):
            new[:, b * c["K"] + k, :, :length] = old[:, b * c["K"] + p, :, :length]
    return new if c["x"] != "u8" else None
