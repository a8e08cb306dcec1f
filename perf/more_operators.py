"""What a decode step does between the logits and the next hidden rows, operator by operator: inputs, plain forms and sizes.

  adjust    orpo_logits_adjust: penalties for repeated tokens, biases and grammar masks, in place on the logits
  history   orpo_beam_history:  the beams' token histories follow their parents and get the new tokens
  advance   orpo_pages_advance, orpo_pages_copy: states in shared pages follow their parents, and the next position is made
            writable: a new page, or a copy of one that other beams hold too
  turnover  orpo_pages_release, orpo_pages_advance: finished sequences let go of their pages, new prompts get theirs
  compact   orpo_pages_compact, orpo_pages_copy: pages in use move to the lowest numbers

Head sizes are those of the recipes in workloads/ (tiny, small, e4b, largev, ragged).
"""

import math
import random

import torch

own = False

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
TYPES = {"fp32": F32, "bf16": BF16, "u8": torch.uint8}
NINF = float("-inf")


def listed():
    return [
        # one prompt, four beams, a short history: latency
        dict(name="adjust tiny", op="adjust", B=1, K=4, V=4096, x="fp32", pad=0, T=128, longest=100, rep=1.2, presence=0.0, frequency=0.0,
             ngram=0, bias=0, masks=0),
        # four prompts on the e4b head with everything on: all three penalties, no repeated trigram, a bias list, a grammar
        dict(name="adjust e4b", op="adjust", B=4, K=4, V=262144, x="fp32", pad=0, T=2048, longest=2000, rep=1.1, presence=0.2, frequency=0.1,
             ngram=3, bias=32, masks=16),
        # a large batch with wide beams, long histories, 16-bit logits, every row under some state of a grammar
        dict(name="adjust largev wide", op="adjust", B=32, K=8, V=128256, x="bf16", pad=0, T=4096, longest=4096, rep=1.1, presence=0.0,
             frequency=0.0, ngram=0, bias=0, masks=64),
        # odd sizes and row pitch
        dict(name="adjust odd", op="adjust", B=7, K=5, V=50257, x="fp32", pad=3, T=777, longest=601, rep=1.3, presence=0.5, frequency=0.0,
             ngram=2, bias=17, masks=5),
        # a short answer of one prompt: latency
        dict(name="history tiny", op="history", B=1, K=4, T=128, longest=100, sources=3),
        # a large batch with wide beams and long answers
        dict(name="history wide", op="history", B=32, K=8, T=8192, longest=8191, sources=5),
        # a short cache of one prompt: latency
        dict(name="advance tiny", op="advance", N=4, B=1, K=4, R=2, page=16, D=64, x="bf16", longest=100, shared=0.5, sources=2),
        # the caches of sixteen layers (keys and values), wide beams that share most of their past
        dict(name="advance cache", op="advance", N=32, B=16, K=8, R=4, page=32, D=128, x="bf16", longest=2040, shared=0.75, sources=4),
        # a few sequences, a quarter of which end
        dict(name="turnover small", op="turnover", B=24, page=16, longest=500, ended=0.25),
        # a serving batch of long sequences in a pool of a hundred thousand pages
        dict(name="turnover large", op="turnover", B=256, page=16, longest=8192, ended=0.25),
        # a small pool, heads of 36, odd page size
        dict(name="compact ragged", op="compact", N=6, B=11, R=3, page=9, D=36, x="bf16", longest=300, live=0.5),
        # 2 GB of keys and values of which two fifths are in use
        dict(name="compact cache", op="compact", N=16, B=64, R=4, page=32, D=128, x="bf16", longest=1100, live=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["adjust", "adjust", "history", "advance", "turnover", "compact"])
    while op == "adjust":
        B, K, V, T = _log(rng, 1, 32), rng.randint(1, 16), _log(rng, 1000, 262144), _log(rng, 16, 16384)
        if B * K * V <= 32 * 8 * 128256 and B * K * T <= 32 * 8 * 4096:
            return dict(op=op, B=B, K=K, V=V, x=rng.choice(["fp32", "bf16"]), pad=rng.choice([0, 0, 1, 8]), T=T, longest=rng.randint(1 + T // 2, T),
                        rep=rng.choice([1.0, 1.1, 1.3]), presence=rng.choice([0.0, 0.4]), frequency=rng.choice([0.0, 0.1]),
                        ngram=rng.choice([0, 0, 2, 3, 4]), bias=rng.choice([0, 0, rng.randint(1, 300)]), masks=rng.choice([0, 0, rng.randint(1, 64)]))
    while op == "history":
        B, K, T = _log(rng, 1, 64), rng.randint(1, 16), _log(rng, 32, 16384)
        if B * K * T <= 32 * 8 * 8192:
            return dict(op=op, B=B, K=K, T=T, longest=rng.randint(1 + T // 2, T - 1), sources=rng.randint(1, K))
    while op == "advance":
        N, B, K, R = _log(rng, 2, 32), _log(rng, 1, 32), rng.randint(2, 10), rng.randint(1, 8)
        page, D, longest = rng.choice([8, 16, 32, 64, 20]), rng.choice([32, 64, 80, 128, 256, 36, 33]), _log(rng, 64, 8192)
        c = dict(op=op, N=N, B=B, K=K, R=R, page=page, D=D, x=rng.choice(["bf16", "bf16", "fp32", "u8"]), longest=longest,
                 shared=round(rng.random(), 2), sources=rng.randint(1, K))
        if work(c)["bytes"] <= 70e6 and N * _pages(c) * R * page * D <= 32 * 2500 * 4 * 32 * 128:
            return c
    while op == "turnover":
        B, longest, page = _log(rng, 1, 512), _log(rng, 64, 32768), rng.choice([8, 16, 32, 64, 20])
        if B * longest / page <= 256 * 8192 / 16:
            return dict(op=op, B=B, page=page, longest=longest, ended=rng.choice([0.1, 0.25, 0.5, 1.0]))
    while True:
        N, B, R, page, D = _log(rng, 2, 32), _log(rng, 1, 128), rng.randint(1, 8), rng.choice([8, 16, 32, 64, 20]), rng.choice([32, 64, 80, 128, 256, 36, 33])
        c = dict(op=op, N=N, B=B, R=R, page=page, D=D, x=rng.choice(["bf16", "bf16", "fp32", "u8"]), longest=_log(rng, 64, 4096),
                 live=round(rng.uniform(0.2, 0.9), 2))
        if N * _pages(c) * R * page * D * 2 <= 2**31:
            return c


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _lengths(c):
    """Spread over the upper half of the longest: the same ones for every seed, in another order."""
    return [c["longest"] - (c["longest"] // 2) * b // c["B"] for b in range(c["B"])]


def _used(c):
    """(columns in use, of them shared by all beams) of each entry."""
    return [(-(-n // c["page"]), int(c.get("shared", 0) * (n // c["page"]))) for n in _lengths(c)]


def _live(c):
    K = c.get("K", 1)
    return sum(s + K * (n - s) for n, s in _used(c))


def _pages(c):
    """Pages of the pool: what is in use and room for one step, for a new set of prompts, or what the case says."""
    if c["op"] == "advance":
        return _live(c) * 5 // 4 + c["B"] * c["K"]
    if c["op"] == "turnover":
        return c["B"] * -(-c["longest"] // c["page"]) * 5 // 4
    return max(2, int(_live(c) / c["live"]))


def _parents(c, r):
    """Per entry, `sources` beams have children, each at least one."""
    rows = []
    for _ in range(c["B"]):
        src = r.sample(range(c["K"]), c["sources"])
        p = src + [r.choice(src) for _ in range(c["K"] - len(src))]
        r.shuffle(p)
        rows.append(p)
    return torch.tensor(rows, dtype=I32, device="cuda")


def _table(c, lens, g):
    """Page table [B * K, columns] on random pages, and how often each page is held."""
    K, pages, dev = c.get("K", 1), _pages(c), "cuda"
    columns = -(-c["longest"] // c["page"]) + 1
    at, beam = torch.arange(columns, device=dev)[None, None], torch.arange(K, device=dev)[None, :, None]
    n = torch.tensor([-(-x // c["page"]) for x in lens], device=dev)[:, None, None]
    s = torch.tensor([int(c.get("shared", 0) * (x // c["page"])) for x in lens], device=dev)[:, None, None]
    first = (at < n) & ((at >= s) | (beam == 0))
    number = (first.reshape(-1).cumsum(0) - 1).view(first.shape)
    number = torch.where(at < s, number[:, :1], number)
    order = torch.randperm(pages, generator=g, device=dev)
    table = torch.where(at < n, order[number.clamp(0, pages - 1)], -1).to(I32).view(c["B"] * K, columns)
    held = torch.zeros(pages + 1, dtype=I32, device=dev).scatter_add_(0, torch.where(table < 0, pages, table).view(-1).long(), torch.ones(table.numel(), dtype=I32, device=dev))
    return table, held[:pages].contiguous()


def _pool(c, g):
    shape = (c["N"], _pages(c), c["R"], c["page"], c["D"])
    if c["x"] == "u8":
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    pool = torch.empty(shape, dtype=TYPES[c["x"]], device="cuda")
    for i in range(c["N"]):
        pool[i] = torch.randn(shape[1:], generator=g, device="cuda")
    return pool


def _ints(values):
    return torch.tensor(values, dtype=I32, device="cuda")


def _ended(c):
    return max(1, int(c["ended"] * c["B"]))


def prepare(case, seed):
    c, g, dev, r = case, _gen(seed), "cuda", random.Random(seed)
    status = torch.zeros(1, dtype=I32, device=dev)
    s = dict(c=c, status=status)
    lens = _lengths(c)
    r.shuffle(lens)
    s["length"] = _ints(lens)
    if c["op"] == "adjust":
        B, K, V, T = c["B"], c["K"], c["V"], c["T"]
        s["logits"] = (torch.randn((B * K, V + c["pad"]), generator=g, device=dev) * 2.5).to(TYPES[c["x"]])[:, :V]
        # frequent tokens come again and again, most only once
        s["history"] = (torch.rand((B * K, T), generator=g, device=dev) ** 3 * V).clamp_(max=V - 1).to(I32)
        s["prompt"] = _ints([n // 4 for n in lens])
        s["bias_token"] = s["bias_value"] = s["masks"] = s["mask_row"] = None
        if c["bias"]:
            start = torch.randint(0, V, (B, 1), generator=g, device=dev)
            s["bias_token"] = ((start + torch.arange(c["bias"], device=dev) * (V // c["bias"])) % V).to(I32)
            s["bias_value"] = torch.randn((B, c["bias"]), generator=g, device=dev) * 4.0
        if c["masks"]:
            # states of a grammar: one that takes few tokens, one that takes all but a few, one in between, and so on
            words = -(-V // 32)
            kind = torch.arange(c["masks"], device=dev)[:, None] % 3
            take = torch.rand((c["masks"], words * 32), generator=g, device=dev)
            take = torch.where(kind == 0, take < 64 / V, torch.where(kind == 1, take >= 64 / V, take < 0.5))
            take = take.view(c["masks"], words, 32).long() << torch.arange(32, device=dev)
            take = take.sum(-1)
            s["masks"] = torch.where(take >= 2**31, take - 2**32, take).to(I32)
            rows = [i % (c["masks"] + 1) - 1 for i in range(B * K)]
            r.shuffle(rows)
            s["mask_row"] = _ints(rows)
    elif c["op"] == "history":
        s["history"] = torch.randint(0, 128256, (c["B"] * c["K"], c["T"]), generator=g, device=dev, dtype=I32)
        s["parent"] = _parents(c, r)
        s["token"] = torch.randint(0, 128256, (c["B"], c["K"]), generator=g, device=dev, dtype=I32)
    else:
        s["table"], s["refs"] = _table(c, lens, g)
        pages, rows = s["refs"].numel(), s["table"].shape[0]
        s["moves"] = torch.zeros((max(rows, pages // 2), 3), dtype=I32, device=dev)
        s["n_moves"] = torch.zeros(1, dtype=I32, device=dev)
        s["ws"] = torch.empty(16 * pages + 64 * rows * s["table"].shape[1] + 65536, dtype=torch.uint8, device=dev)
        if c["op"] == "turnover":
            ends = [i < _ended(c) for i in range(c["B"])]
            r.shuffle(ends)
            new = _lengths(c)
            r.shuffle(new)
            s["ended"] = torch.tensor(ends, dtype=torch.uint8, device=dev)
            s["length"] = _ints([0 if e else n for e, n in zip(ends, lens)])  # of what goes on
            s["more"] = _ints([n if e else 0 for e, n in zip(ends, new)])  # the new prompts
        else:
            s["pool"] = _pool(c, g)
            if c["op"] == "advance":
                s["parent"] = _parents(c, r)
            else:
                s["new_table"], s["new_refs"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
                s["live"] = torch.zeros(1, dtype=I32, device=dev)
    return s


def run(state):
    op = state["c"]["op"]
    return {"adjust": _adjust, "history": _history, "advance": _advance, "turnover": _turnover, "compact": _compact}[op](state)


def _adjust(s):
    c, logits, history = s["c"], s["logits"], s["history"]
    if own:
        import orpo_preference_loss_gb300 as orpo
        orpo.orpo_logits_adjust(logits, c["K"], s["status"], history, s["length"], s["prompt"], c["rep"], c["presence"], c["frequency"], c["ngram"],
                                s["bias_token"], s["bias_value"], s["masks"], s["mask_row"])
        return logits
    V, K, T = c["V"], c["K"], history.shape[1]
    x = logits.float()
    at = torch.arange(T, device=x.device)[None]
    length, prompt = s["length"].repeat_interleave(K)[:, None], s["prompt"].repeat_interleave(K)[:, None]
    token = torch.where(at < length, history, V).long()
    seen = torch.zeros((x.shape[0], V + 1), dtype=torch.bool, device=x.device).scatter_(1, token, True)[:, :V]
    count = torch.zeros((x.shape[0], V + 1), device=x.device).scatter_add_(1, token, (at >= prompt).float())[:, :V]
    if c["rep"] != 1:
        x = torch.where(seen, torch.where(x > 0, x / c["rep"], x * c["rep"]), x)
    x = x - (c["presence"] * (count > 0) + c["frequency"] * count)
    if c["bias"]:
        row = torch.zeros((c["B"], V), device=x.device).scatter_add_(1, s["bias_token"].long(), s["bias_value"])
        x = x + row.repeat_interleave(K, 0)
    n = c["ngram"]
    if n and T >= n:
        tail = length - (n - 1) + torch.arange(n - 1, device=x.device)[None]
        same = (history.unfold(1, n, 1)[:, :, :n - 1] == history.gather(1, tail.clamp(min=0).long())[:, None]).all(-1)
        same &= at[:, n - 1:] < length
        ban = torch.zeros((x.shape[0], V + 1), dtype=torch.bool, device=x.device)
        ban.scatter_(1, torch.where(same, token[:, n - 1:], V), True)
        x = torch.where(ban[:, :V], NINF, x)
    if s["masks"] is not None:
        words = s["masks"][s["mask_row"].clamp(min=0).long()]
        bits = (words[:, :, None] >> torch.arange(32, dtype=I32, device=x.device)) & 1
        bits = bits.view(x.shape[0], -1)[:, :V]
        x = torch.where((bits == 0) & (s["mask_row"] >= 0)[:, None], NINF, x)
    logits.copy_(x)
    return logits


def _history(s):
    c, history = s["c"], s["history"]
    if own:
        import orpo_preference_loss_gb300 as orpo
        orpo.orpo_beam_history(history, s["parent"], s["token"], s["length"], s["status"])
        return history
    v = history.view(c["B"], c["K"], c["T"])
    at = torch.arange(c["T"], device=v.device)[None, None]
    length = s["length"][:, None, None]
    new = v.gather(1, s["parent"].long()[:, :, None].expand(-1, -1, c["T"]))
    v.copy_(torch.where(at < length, new, torch.where(at == length, s["token"][:, :, None], v)))
    return history


def _held(table, pages):
    """How often each page is in a table."""
    held = torch.zeros(pages + 1, dtype=I32, device=table.device)
    return held.scatter_add_(0, torch.where(table < 0, pages, table).view(-1).long(), torch.ones_like(table).view(-1))[:pages]


def _reserve(table, refs, length, more, most, page):
    """Makes positions length .. length + more - 1 of each row writable. Returns (old pages, new pages) of the items [rows, items of a row]
    and the positions to copy from old to new."""
    pages, dev = refs.numel(), table.device
    width = (most - 1 + page - 1) // page + 1
    begin = length // page
    at = begin[:, None] + torch.arange(width, device=dev)[None]
    inside = (at < ((length + more + page - 1) // page)[:, None]) & (more > 0)[:, None]
    at = at.clamp(max=table.shape[1] - 1).long()
    old = table.gather(1, at)
    item = torch.arange(old.numel(), dtype=I32, device=dev).view(old.shape)
    # of the rows that hold a page together the last keeps it, if nothing else holds it
    slot = torch.where(inside & (old >= 0), old, pages).long()
    count = torch.zeros(pages + 1, dtype=I32, device=dev).scatter_add_(0, slot.view(-1), torch.ones_like(item).view(-1))
    last = torch.full((pages + 1,), -1, dtype=I32, device=dev).scatter_reduce_(0, slot.view(-1), item.view(-1), "amax")
    held = torch.cat((refs, refs.new_zeros(1)))
    shared = (held[slot] > 1) & ~((held[slot] == count[slot]) & (last[slot] == item))
    need = inside & ((old < 0) | shared)
    free = refs == 0
    order = torch.full((pages + 1,), -1, dtype=I32, device=dev)
    order.scatter_(0, torch.where(free, free.cumsum(0) - 1, pages), torch.arange(pages, dtype=I32, device=dev))
    rank = (need.view(-1).cumsum(0) - 1).view(need.shape).clamp(min=0)
    fresh = torch.where(need, order[rank], old)
    one = need.to(I32).view(-1)
    refs.add_(torch.zeros(pages + 1, dtype=I32, device=dev).scatter_add_(0, torch.where(need, fresh, pages).long().view(-1), one)[:pages])
    gone = need & (old >= 0)
    refs.sub_(torch.zeros(pages + 1, dtype=I32, device=dev).scatter_add_(0, torch.where(gone, old, pages).long().view(-1), one)[:pages])
    # items that are not inside write to a column of their own
    wide = torch.cat((table, table.new_zeros((table.shape[0], 1))), 1)
    wide.scatter_(1, torch.where(inside, at, table.shape[1]), fresh)
    table.copy_(wide[:, :-1])
    filled = torch.where(gone & (at == begin[:, None]), (length % page)[:, None], 0)
    return old, fresh, filled


def _advance(s):
    c, table, refs, pool = s["c"], s["table"], s["refs"], s["pool"]
    if own:
        import orpo_preference_loss_gb300 as orpo
        orpo.orpo_pages_advance(table, refs, c["page"], s["parent"], s["length"], None, 1, s["moves"], s["n_moves"], s["ws"], s["status"])
        orpo.orpo_pages_copy(pool, s["moves"], s["n_moves"], s["status"])
        return [table, refs, pool]
    B, K, page = c["B"], c["K"], c["page"]
    v = table.view(B, K, -1)
    took = v.gather(1, s["parent"].long()[:, :, None].expand_as(v))
    used = torch.arange(v.shape[2], device=v.device)[None, None] < ((s["length"] + page - 1) // page)[:, None, None]
    new = torch.where(used, took, v)
    refs.add_(_held(new, refs.numel()) - _held(v, refs.numel()))
    v.copy_(new)
    length = s["length"].repeat_interleave(K)
    old, fresh, filled = _reserve(table, refs, length, torch.ones_like(length), 1, page)
    dst = fresh.view(-1).long()
    src = torch.where(filled.view(-1) > 0, old.view(-1), fresh.view(-1)).long()
    moves = torch.arange(page, device=v.device)[None] < filled.view(-1, 1)
    pool[:, dst] = torch.where(moves[None, :, None, :, None], pool[:, src], pool[:, dst])
    return [table, refs, pool]


def _turnover(s):
    c, table, refs = s["c"], s["table"], s["refs"]
    if own:
        import orpo_preference_loss_gb300 as orpo
        orpo.orpo_pages_release(table, refs, s["ended"], s["status"])
        orpo.orpo_pages_advance(table, refs, c["page"], None, s["length"], s["more"], c["longest"], s["moves"], s["n_moves"], s["ws"], s["status"])
        return [table, refs]
    left = torch.where(s["ended"][:, None] != 0, -1, table)
    refs.add_(_held(left, refs.numel()) - _held(table, refs.numel()))
    table.copy_(left)
    _reserve(table, refs, s["length"], s["more"], c["longest"], c["page"])
    return [table, refs]


def _compact(s):
    c, table, refs, pool = s["c"], s["table"], s["refs"], s["pool"]
    if own:
        import orpo_preference_loss_gb300 as orpo
        orpo.orpo_pages_compact(table, refs, c["page"], s["new_table"], s["new_refs"], s["live"], s["moves"], s["n_moves"], s["ws"], s["status"])
        orpo.orpo_pages_copy(pool, s["moves"], s["n_moves"], s["status"])
        return [s["new_table"], s["new_refs"], s["live"], pool]
    pages, dev = refs.numel(), refs.device
    used = refs > 0
    n = used.sum()
    number = torch.arange(pages, device=dev)
    hole, mover = ~used & (number < n), used & (number >= n)
    half = pages // 2
    # the i-th hole and the i-th page that moves; where there are no more, a page in use "moves" to its own place
    stay = torch.argmax(used.to(I32))
    holes = stay.expand(half + 1).scatter(0, torch.where(hole, hole.cumsum(0) - 1, half), number)[:half]
    movers = stay.expand(half + 1).scatter(0, torch.where(mover, mover.cumsum(0) - 1, half), number)[:half]
    to = torch.where(used, number, 0).scatter(0, movers, holes).to(I32)
    s["new_table"].copy_(torch.where(table < 0, -1, to[table.clamp(min=0).long()]))
    s["new_refs"].copy_(torch.where(mover, 0, refs).scatter(0, holes, refs[movers]))
    s["live"].copy_(n)
    pool[:, holes] = pool[:, movers]
    return [s["new_table"], s["new_refs"], s["live"], pool]


def _distinct(n, V):
    """Different tokens among n of floor(V u^3), u uniform: the sum over tokens of 1 - exp(-n p)."""
    return sum(3 * V * u * u * (1 - math.exp(-n / (3 * V * u * u))) for u in ((i + 0.5) / 256 for i in range(256))) / 256


def work(case):
    c = case
    lens = _lengths(c)
    K = c.get("K", 1)
    if c["op"] == "adjust":
        V, T, size, rows = c["V"], sum(lens) * K, {"fp32": 4, "bf16": 2}[c["x"]], c["B"] * K
        touched = 0
        if c["rep"] != 1 or c["presence"] or c["frequency"]:
            touched = K * sum(_distinct(n, V) for n in lens)
        history = 4 * T if touched or c["ngram"] else 0
        masked = 0.0
        if c["masks"]:
            rate = [(1 - 64 / V, 64 / V, 0.5)[m % 3] for m in range(c["masks"])]
            masked = V * sum(rate[i % (c["masks"] + 1) - 1] for i in range(rows) if i % (c["masks"] + 1))
        bits = min(c["masks"], rows) * -(-V // 32) * 4
        return {"bytes": history + bits + c["B"] * c["bias"] * 8 + size * (2 * (touched + rows * c["bias"]) + masked), "flops": 4 * touched + T}
    if c["op"] == "history":
        # a random map leaves one beam its own on average
        return {"bytes": 4 * sum(lens) * (K - 1 + min(c["sources"], K - 1)) + 12 * c["B"] * K, "flops": 0}
    columns = K * sum(n for n, _ in _used(c))
    pages = _pages(c)
    if c["op"] == "turnover":
        share = _ended(c) / c["B"]
        return {"bytes": 4 * (pages + 4 * columns * share), "flops": 0}
    size = {"fp32": 4, "bf16": 2, "u8": 1}[c["x"]]
    if c["op"] == "advance":
        positions = (K - c["sources"]) * sum(n % c["page"] for n in lens)
        return {"bytes": 4 * (pages + 2 * columns) + 2 * c["N"] * c["R"] * c["D"] * size * positions, "flops": 0}
    live = _live(c)
    moved = live * (pages - live) // pages
    return {"bytes": 8 * (pages + columns) + 2 * c["N"] * c["R"] * c["page"] * c["D"] * size * moved, "flops": 0}


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "adjust":
        x = s["logits"].double()
        history, lens, prompts = s["history"].cpu(), s["length"].tolist(), s["prompt"].tolist()
        for r in range(x.shape[0]):
            b = r // c["K"]
            h = history[r, :lens[b]].long()
            seen = torch.bincount(h, minlength=c["V"]).cuda() > 0
            n = torch.bincount(h[min(prompts[b], lens[b]):], minlength=c["V"]).cuda().double()
            y = x[r]
            y[seen & (y > 0)] /= c["rep"]
            y[seen & (s["logits"][r] <= 0)] *= c["rep"]
            y -= n.clamp(max=1) * c["presence"] + n * c["frequency"]
            if c["bias"]:
                y[s["bias_token"][b].long()] += s["bias_value"][b].double()
            k = c["ngram"]
            if k and lens[b] >= k:
                words = h.tolist()
                end = words[len(words) - k + 1:]
                y[[words[i + k - 1] for i in range(len(words) - k + 1) if words[i:i + k - 1] == end]] = NINF
            if c["masks"] and int(s["mask_row"][r]) >= 0:
                mask = s["masks"][int(s["mask_row"][r])].long()
                v = torch.arange(c["V"], device=x.device)
                y[(mask[v // 32] >> (v % 32)) % 2 == 0] = NINF
        return x
    if c["op"] in ("history", "turnover"):
        return None
    table, refs, page = s["table"].tolist(), s["refs"].tolist(), c["page"]
    pool = s["pool"].double() if c["x"] != "u8" else None
    if pool is None or pool.numel() > 2**31:
        return None
    if c["op"] == "advance":
        lens = s["length"].tolist()
        before = [row[:] for row in table]
        for b, parents in enumerate(s["parent"].tolist()):
            for k, p in enumerate(parents):
                n = -(-lens[b] // page)
                table[b * c["K"] + k][:n] = before[b * c["K"] + p][:n]
        refs = [0] * len(refs)
        for row in table:
            for e in row:
                if e >= 0:
                    refs[e] += 1
        free = [p for p, n in enumerate(refs) if n == 0]
        for r, row in enumerate(table):
            at, fill = divmod(lens[r // c["K"]], page)
            if row[at] < 0 or refs[row[at]] > 1:
                new = free.pop(0)
                if row[at] >= 0:
                    refs[row[at]] -= 1
                    pool[:, new, :, :fill] = pool[:, row[at], :, :fill]
                row[at] = new
        return [None, None, pool]
    live = sum(n > 0 for n in refs)
    holes = [p for p in range(live) if refs[p] == 0]
    movers = [p for p in range(live, len(refs)) if refs[p] > 0]
    pool[:, holes] = pool[:, movers]
    return [None, None, None, pool]
