"""Workloads of rotary positions and of eviction from the quantized key/value cache.

A model that serves long texts rotates its queries and keys by their positions
before the keys are quantized into the cache, sums up how much attention each
cached token gets, and, once a context outgrows its budget, keeps the tokens
that got most.  Each case is one pass through one of these operators at sizes
of real serving.  The head layout of most cases (32 query heads over 8 cache
heads of 128 channels) is that of the models whose projections this package
benchmarks; the rest are generic.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
BASE = 1e6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the angles of one decode step's tokens, made once a step for all layers (latency)
        {"name": "table_step_32", "op": "table", "rows": 32, "rot": 128, "range": False},
        # a model's whole table, made when it is loaded
        {"name": "table_131072", "op": "table", "rows": 131072, "rot": 128, "range": True},
        # queries and keys of a decode step, side by side in the fused projection's rows
        {"name": "rotate_step_32", "op": "rotate", "tokens": 32, "heads": 40, "dim": 128, "rot": 128,
         "interleaved": False, "backward": False, "rows": 32768},
        # gradients of a training batch's queries: half of each head rotated, neighbouring channels paired
        {"name": "rotate_backward_8001", "op": "rotate", "tokens": 8001, "heads": 32, "dim": 96, "rot": 48,
         "interleaved": True, "backward": True, "rows": 8192},
        # one decode step of 64 sequences: queries rotated, keys rotated and stored, values stored
        {"name": "append_step_64", "op": "append", "tokens": 64, "qheads": 32, "heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "bits": 4, "page": 64, "holes": False, "rows": 131072},
        # a long prompt, the same, out of the fused qkv projection; a fifth of the padded batch has no slot
        {"name": "append_prompt_8192", "op": "append", "tokens": 8192, "qheads": 32, "heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "bits": 4, "page": 64, "holes": True, "rows": 32768},
        # one user, one token, a short context: launch and latency
        {"name": "weigh_1x517", "op": "weigh", "batch": 1, "kv": 517, "nq": 1, "qheads": 32, "heads": 8, "dim": 128,
         "bits": 4, "page": 64, "window": 0, "ragged": False, "sum": True},
        # a decode batch, full contexts: each step adds to what the tokens have gathered
        {"name": "weigh_96x16384", "op": "weigh", "batch": 96, "kv": 16384, "nq": 1, "qheads": 32, "heads": 8,
         "dim": 128, "bits": 4, "page": 64, "window": 0, "ragged": False, "sum": True},
        # the last tokens of freshly read prompts decide what is kept of them
        {"name": "weigh_last_16x64", "op": "weigh", "batch": 16, "kv": 8191, "nq": 64, "qheads": 16, "heads": 16,
         "dim": 64, "bits": 8, "page": 32, "window": 0, "ragged": True, "sum": False},
        # prompt chunks over what is already cached and themselves
        {"name": "weigh_prompt_2x2048", "op": "weigh", "batch": 2, "kv": 8192, "nq": 2048, "qheads": 32, "heads": 8,
         "dim": 128, "bits": 4, "page": 64, "window": 0, "ragged": False, "sum": True},
        # one context of odd length cut to half
        {"name": "evict_1x2001_8bit", "op": "evict", "batch": 1, "kv": 2001, "budget": 1000, "first": 4, "last": 129,
         "heads": 16, "dim": 64, "bits": 8, "page": 16, "ragged": False},
        # a batch of long contexts cut to an eighth
        {"name": "evict_32x16384", "op": "evict", "batch": 32, "kv": 16384, "budget": 2048, "first": 4, "last": 256,
         "heads": 8, "dim": 128, "bits": 4, "page": 64, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["table", "rotate", "append", "weigh", "weigh", "weigh", "evict", "evict"])
    dim, bits, page = rng.choice([64, 128, 128]), rng.choice([4, 4, 8]), rng.choice([16, 32, 64, 128, 256])
    rows = rng.choice([8192, 32768, 131072])
    if kind == "table":
        return {"op": "table", "rows": _log(rng, 1, 131072), "rot": rng.choice([16, 32, 48, 64, 96, 128]),
                "range": rng.random() < 0.5}
    if kind == "rotate":
        heads, dim = rng.choice([1, 2, 5, 8, 16, 32, 40]), rng.choice([64, 80, 96, 128, 256])
        return {"op": "rotate", "tokens": _log(rng, 1, min(16384, 8192 * 32 * 96 // (heads * dim))), "heads": heads,
                "dim": dim, "rot": rng.choice([16, 32, dim // 2, dim]), "interleaved": rng.random() < 0.5,
                "backward": rng.random() < 0.5, "rows": rows}
    if kind == "append":
        heads, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 7])
        most = 8192 * 48 * 128 // (heads * (group + 2) * dim)
        return {"op": "append", "tokens": _log(rng, 1, min(most, 16384)), "qheads": heads * group, "heads": heads,
                "dim": dim, "rot": rng.choice([32, dim // 2, dim, dim]), "interleaved": rng.random() < 0.4,
                "bits": bits, "page": page, "holes": rng.random() < 0.5, "rows": rows}
    heads = rng.choice([1, 2, 4, 5, 8, 16])
    if kind == "evict":
        batch = _log(rng, 1, 64)
        kv = _log(rng, 64, min(65536, 32 * 16384 * 8 // (2 * batch * heads)))
        budget = _log(rng, 16, min(kv, 32 * 2048 * 8 // (batch * heads)))
        first = rng.choice([0, 1, 4])
        return {"op": "evict", "batch": batch, "kv": kv, "budget": budget, "first": first,
                "last": rng.randint(0, budget - first), "heads": heads, "dim": dim, "bits": bits, "page": page,
                "ragged": rng.random() < 0.6}
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if rng.random() < 0.6:  # single tokens or a few drafted ones
        nq = rng.choice([1, 1, 1, 2, 4, 7])
        batch = _log(rng, 1, 96)
        kv = _log(rng, max(nq, 100), min(131072, max(256, 96 * 16384 * 8 // (2 * batch * heads * group))))
    else:  # prompts, or their last tokens
        nq = _log(rng, 16, 2048)
        batch = _log(rng, 1, 8)
        kv = nq + _log(rng, 1, 6144)
        while batch * nq * kv * heads * group > 2 * 2048 * 8192 * 32:
            batch, nq = max(1, batch // 2), max(16, nq // 2)
    return {"op": "weigh", "batch": batch, "kv": kv, "nq": nq, "qheads": heads * group, "heads": heads, "dim": dim,
            "bits": bits, "page": page, "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
            "ragged": rng.random() < 0.6, "sum": rng.random() < 0.6}


def _lengths(case):
    """Cache length and query tokens of each sequence: part of the case, the same for every seed."""
    b, kv, nq = case["batch"], case["kv"], case.get("nq", 1)
    if not case["ragged"]:
        return [kv] * b, [nq] * b
    r = random.Random("%d %d %d" % (b, kv, nq))
    lens = [kv] + [r.randint(1, kv) for _ in range(b - 1)]
    qs = [nq] + [r.randint(1, nq) for _ in range(b - 1)]
    return lens, [min(q, n) for q, n in zip(qs, lens)]


def _row_bytes(case):
    return case["dim"] * case["bits"] // 8 + 4  # codes, scale and low value of one token of one head


def work(case):
    op = case["op"]
    if op == "table":
        n, r = case["rows"], case["rot"]
        return {"bytes": 4 * n * r + 4 * r + (0 if case["range"] else 8 * n), "flops": 2 * n * r}
    if op == "rotate":
        t, h, d, r = case["tokens"], case["heads"], case["dim"], case["rot"]
        return {"bytes": 4 * t * h * d + 4 * t * r + 8 * t, "flops": 3 * t * h * r}
    if op == "append":  # rotated and written, then the keys and values read back
        t, h, d, r = case["tokens"], case["heads"], case["dim"], case["rot"]
        full, packed = 2 * t * h * d * 2, 2 * t * h * _row_bytes(case)
        return {"bytes": 4 * t * case["qheads"] * d + 2 * full + 2 * packed + 4 * t * r + 24 * t,
                "flops": 3 * t * (case["qheads"] + h) * r + 6 * full}
    lens, qs = _lengths(case)
    h = case["heads"]
    if op == "evict":  # chosen and moved, then the keys and values read back
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": 4 * sum(lens) * h + kept * h * (6 * _row_bytes(case) + 4 + 4 + 4 * case["dim"]),
                "flops": sum(lens) * h + 4 * kept * h * case["dim"]}
    w = case["window"]
    pairs, seen = 0, 0
    for n, q in zip(lens, qs):
        first = n - q  # position of the first query
        if w:
            pairs += sum(min(p + 1, w) for p in range(first, n))
            seen += n - max(0, first + 1 - w)
        else:
            pairs += q * first + q * (q + 1) // 2
            seen += n
    return {"bytes": seen * h * _row_bytes(case) + 2 * sum(qs) * case["qheads"] * case["dim"] +
            4 * seen * h * (2 if case["sum"] else 1) + 4 * seen // case["page"],
            "flops": (2 * case["dim"] + 2) * pairs * case["qheads"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _heads(g, tokens, heads, dim, spread):
    """bf16 rows ~ N(0, 1) with a few channels `spread` times as large, as keys have them."""
    x = torch.randn((tokens, heads, dim), generator=g, device=DEV)
    gain = torch.ones((heads, dim), device=DEV)
    gain.view(-1)[torch.randint(0, heads * dim, (max(1, heads * dim // 32),), generator=g, device=DEV)] = spread
    return (x * gain).to(torch.bfloat16)


def _freqs(rot):
    """Radians a position: BASE ** (-2 i / rot), in 64 bits."""
    return torch.tensor([BASE ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=DEV)


def _positions(g, tokens, rows):
    """Positions of a batch's tokens: runs of neighbours from anywhere in the table."""
    run = 1 + tokens // 8
    at = torch.randint(0, max(1, rows - run), (8,), generator=g, device=DEV)
    t = torch.arange(tokens, device=DEV)
    return (at[t // run] + t % run).clamp(max=rows - 1)


def _random_cache(g, pages, heads, page, dim, bits):
    codes = torch.randint(0, 256, (pages, 2, heads, page, dim * bits // 8), generator=g, device=DEV,
                          dtype=torch.uint8)
    params = torch.rand((pages, 2, heads, page, 2), generator=g, device=DEV)
    params[..., 1] = -params[..., 1] * (2 ** bits - 1) / 2
    return codes, params.to(torch.bfloat16)


def _pages(g, lens, page, spare):
    """A page table of sequences whose pages lie anywhere (-1 where there is none), and the pool's size."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = table.to(DEV)
    return torch.where(table >= 0, order[table.clamp(min=0).long()], table), order, need


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "table":
        s = {"case": case, "freqs": _freqs(case["rot"])}
        if case["range"]:
            s["positions"] = case["rows"]
            s["freqs"] *= 0.5 + torch.rand((), generator=g, device=DEV, dtype=torch.float64)  # a model's own base
        else:
            s["positions"] = torch.randint(0, 1 << 20, (case["rows"],), generator=g, device=DEV)
        return s
    if op in ("rotate", "append"):
        t, rows = case["tokens"], case["rows"]
        angles = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * _freqs(case["rot"])
        s = {"case": case, "positions": _positions(g, t, rows),
             "table": torch.cat([torch.cos(angles), torch.sin(angles)], 1).float()}
        if op == "rotate":
            h = case["heads"]
            # a slice of a fused projection's rows
            s["x"] = _heads(g, t, h + 8, case["dim"], 8.0)[:, :h]
            return s
    d, bits, page, heads = case["dim"], case["bits"], case["page"], case["heads"]
    if op == "append":
        pages = -(-t // page) + 3
        order = torch.randperm(pages, generator=g, device=DEV)[: -(-t // page)]
        slots = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:t].contiguous()
        if case["holes"]:
            slots[torch.rand(t, generator=g, device=DEV) < 0.2] = -1
        s["slots"] = slots
        s["codes"], s["params"] = _random_cache(g, pages, heads, page, d, bits)
        hq = case["qheads"]
        s["qkv"] = torch.cat([_heads(g, t, hq, d, 4.0), _heads(g, t, heads, d, 8.0), _heads(g, t, heads, d, 1.0)], 1)
        return s
    lens, qs = _lengths(case)
    if op == "evict":
        new = [min(n, case["budget"]) for n in lens]
        need = [-(-n // page) for n in new]
        table, order, _ = _pages(g, lens, page, sum(need))
        pages = order.shape[0]
        moved = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
        slots, at = [], pages - sum(need)
        for i, n in enumerate(need):
            moved[i, :n] = torch.arange(at, at + n, dtype=torch.int32)
            slots.append(torch.arange(at * page, at * page + new[i]))
            at += n
        moved = moved.to(DEV)
        slots = torch.cat(slots).to(DEV)
        s = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
             "new_table": torch.where(moved >= 0, order[moved.clamp(min=0).long()], moved),
             "slots": order[slots // page].long() * page + slots % page}
        s["codes"], s["params"] = _random_cache(g, pages, heads, page, d, bits)
        # sums of attention: few tokens got much, a fifth got nothing that 32 bits hold
        w = torch.exp(2.0 * torch.randn((pages, heads, page), generator=g, device=DEV))
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.2, torch.zeros_like(w), w)
        return s
    b = case["batch"]
    table, order, need = _pages(g, lens, page, 1)
    pages = order.shape[0]
    codes = torch.zeros((pages, 2, heads, page, d * bits // 8), dtype=torch.uint8, device=DEV)
    params = torch.zeros((pages, 2, heads, page, 2), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 28) // (heads * page * d))
    for i in range(0, pages, step):  # keys; no value is read
        n = min(step, pages - i)
        x = _heads(g, n * page, heads, d, 4.0).view(n, page, heads, d).transpose(1, 2)
        c, p = _quantize(x.float(), bits)
        codes[i:i + n, 0] = _pack(c, bits)
        params[i:i + n, 0] = p
    # what lies behind a sequence's end in its last page was never written
    for i, n in enumerate(lens):
        if n % page:
            params[order[sum(need[:i + 1]) - 1].long(), :, :, n % page:] = float("nan")
    offsets = torch.zeros(b + 1, dtype=torch.int32)
    offsets[1:] = torch.tensor(qs, dtype=torch.int32).cumsum(0)
    return {"case": case, "q": _heads(g, sum(qs), case["qheads"], d, 1.0), "codes": codes, "params": params,
            "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "offsets": offsets.to(DEV),
            "max_q": max(qs), "weights": torch.zeros((pages, heads, page), device=DEV),
            "previous": torch.rand((pages, heads, page), generator=g, device=DEV) if case["sum"] else None}


# ------------------------------------------------------------------ plain forms

def _quantize(x, bits):
    """Codes and (scale, low) of fp32 rows: the scale is (max - min) / levels rounded up to bf16."""
    levels = 2 ** bits - 1
    lo = x.amin(-1, keepdim=True)
    r = x.amax(-1, keepdim=True) - lo
    r = r / torch.full_like(r, levels)  # a division: dividing by a number would multiply by its inverse
    s = ((r.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)  # r >= 0
    c = torch.where(s > 0, torch.round((x - lo) / s), torch.zeros_like(x)).clamp(0, levels)
    return c.to(torch.uint8), torch.cat([s, lo], -1).to(torch.bfloat16)


def _pack(c, bits):
    return c if bits == 8 else c[..., 0::2] | (c[..., 1::2] << 4)


def _unpack(codes, bits):
    return codes if bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def _values(codes, params, bits):
    """fp32 values of packed rows."""
    p = params.float()
    return p[..., 1:] + p[..., :1] * _unpack(codes, bits)


def _read(s):
    """bf16 keys and values [tokens, heads, dim] of the slots; zeros where there is none."""
    page = s["case"]["page"]
    there = s["slots"] >= 0
    at = s["slots"].clamp(min=0)
    x = _values(s["codes"][at // page, :, :, at % page], s["params"][at // page, :, :, at % page], s["case"]["bits"])
    x = torch.where(there[:, None, None, None], x, torch.zeros_like(x)).to(torch.bfloat16)
    return x[:, 0].contiguous(), x[:, 1].contiguous()


def _table(s):
    at = s["positions"]
    if s["case"]["range"]:
        at = torch.arange(at, device=DEV)
    angles = at.double()[:, None] * s["freqs"]
    return torch.cat([torch.cos(angles), torch.sin(angles)], 1).float()


def _rotate(x, rows, interleaved, backward):
    """Pairs of x [tokens, heads, dim] turned by the angles of rows [tokens, rot]."""
    r = rows.shape[1]
    cos, sin = rows[:, None, : r // 2], rows[:, None, r // 2:]
    if backward:
        sin = -sin
    t = x[..., :r].float()
    a, b = (t[..., 0::2], t[..., 1::2]) if interleaved else (t[..., : r // 2], t[..., r // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    t = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([t.to(torch.bfloat16), x[..., r:]], -1)


def _append(s):
    case = s["case"]
    page, bits, hq, h = case["page"], case["bits"], case["qheads"], case["heads"]
    x = _rotate(s["qkv"][:, :hq + h], s["table"][s["positions"]], case["interleaved"], False)
    there = s["slots"] >= 0
    at = s["slots"][there]
    kv = torch.stack([x[:, hq:], s["qkv"][:, hq + h:]], 1)[there].float()
    c, p = _quantize(kv, bits)
    s["codes"][at // page, :, :, at % page] = _pack(c, bits)
    s["params"][at // page, :, :, at % page] = p
    return x[:, :hq].contiguous(), *_read(s)


def _weigh(s):
    """weights = (previous, but 0 for the query tokens themselves) + the softmax weights summed over the rows."""
    case = s["case"]
    b, hq, h, d, page = case["batch"], case["qheads"], case["heads"], case["dim"], case["page"]
    mq, wide = s["max_q"], s["table"].shape[1]
    at = s["table"].clamp(min=0).long()
    lens = s["lens"].long()
    nq = (s["offsets"][1:] - s["offsets"][:-1]).long()
    j = torch.arange(wide * page, device=DEV)
    live = j < lens[:, None]  # [batch, tokens]
    # [batch, pages, heads, page, .] -> [batch, heads, tokens, .]
    flat = lambda x: x.transpose(1, 2).flatten(2, 3)  # noqa: E731
    k = _values(flat(s["codes"][at, 0]), torch.where(live[:, None, :, None], flat(s["params"][at, 0]),
                torch.zeros((), device=DEV, dtype=torch.bfloat16)), case["bits"])
    i = torch.arange(mq, device=DEV)
    row = (s["offsets"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)  # [batch, max_q]
    q = s["q"].float()[row].view(b, mq, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, hq // h * mq, d)
    pos = (lens - nq)[:, None] + i  # [batch, max_q]
    see = (j <= pos[..., None]) & (i < nq[:, None])[..., None]
    if case["window"]:
        see &= j > pos[..., None] - case["window"]
    x = torch.matmul(q, k.transpose(2, 3)).view(b, h, hq // h, mq, -1) * d ** -0.5
    x = torch.where(see[:, None, None], x, torch.full((), float("-inf"), device=DEV))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = x.sum(-1, keepdim=True)
    x = (x / torch.where(total > 0, total, torch.ones_like(total))).sum((2, 3))  # [batch, heads, tokens]
    if case["sum"]:
        older = j < (lens - nq)[:, None]
        x = x + torch.where(older[:, None], flat(s["previous"][at, :, :, None])[..., 0], torch.zeros_like(x))
    # the tokens that some query sees
    seen = see.any(1)
    slot = at[..., None] * page + torch.arange(page, device=DEV)  # [batch, pages, page]
    slot = slot.flatten(1)[seen]
    s["weights"][slot // page, :, slot % page] = x.transpose(1, 2)[seen]
    return s["weights"]


def _evict(s):
    case = s["case"]
    b, h, page, budget = case["batch"], case["heads"], case["page"], case["budget"]
    first, last = case["first"], case["last"]
    at = s["table"].clamp(min=0).long()
    lens = s["lens"].long()
    new = lens.clamp(max=budget)
    j = torch.arange(at.shape[1] * page, device=DEV)
    w = s["weights"][at].transpose(1, 2).flatten(2)  # [batch, heads, tokens]
    safe = (j < first) | (j >= lens[:, None] - last) | (lens[:, None] <= budget)
    live = j < lens[:, None]
    w = torch.where(safe[:, None], torch.full((), float("inf"), device=DEV), w)
    w = torch.where(live[:, None], w, torch.full((), float("-inf"), device=DEV))
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices
    wide = min(budget, w.shape[2])
    kept = best[..., :wide]
    kept = torch.where((torch.arange(wide, device=DEV) < new[:, None])[:, None], kept, w.shape[2])
    kept = torch.sort(kept, -1).values
    there = (torch.arange(wide, device=DEV) < new[:, None])[:, None].expand(b, h, wide)
    i, hh, t = there.nonzero(as_tuple=True)
    src = kept[there]
    to = s["new_table"].long()[i, t // page]
    src_page = at[i, src // page]
    for x in (s["codes"], s["params"]):
        x[to, :, hh, t % page] = x[src_page, :, hh, src % page]
    s["weights"][to, hh, t % page] = s["weights"][src_page, hh, src % page]
    out = torch.full((b, h, budget), -1, dtype=torch.int32, device=DEV)
    out[..., :wide] = torch.where(there, kept, -1).to(torch.int32)
    return new.to(torch.int32), out, s["weights"], *_read(s)


def run(state):
    case, s = state["case"], state
    op = case["op"]
    if own:
        from int8_quantized_linear_gb300 import capi
        if op == "table":
            return capi.rotary_table(s["freqs"], s["positions"])
        if op == "rotate":
            return capi.rotary_apply(s["x"], s["table"], s["positions"], interleaved=case["interleaved"],
                                     backward=case["backward"])
        if op == "append":
            q, k, v = s["qkv"].split([case["qheads"], case["heads"], case["heads"]], dim=1)
            q = capi.kv_cache_store_rotary(q, k, v, s["table"], s["slots"], s["codes"], s["params"],
                                           positions=s["positions"], interleaved=case["interleaved"])
            return q, *capi.kv_cache_load(s["codes"], s["params"], s["slots"], case["dim"])
        if op == "weigh":
            offsets = {} if case["nq"] == 1 else {"q_offsets": s["offsets"], "max_q": s["max_q"]}
            return capi.kv_cache_weights(s["q"], s["codes"], s["params"], s["table"], s["lens"], s["weights"],
                                         previous=s["previous"], window=case["window"], **offsets)
        new, kept = capi.kv_cache_evict(s["codes"], s["params"], s["weights"], s["table"], s["lens"], case["budget"],
                                        first=case["first"], last=case["last"], new_table=s["new_table"])
        return new, kept, s["weights"], *capi.kv_cache_load(s["codes"], s["params"], s["slots"], case["dim"])
    if op == "table":
        return _table(s)
    if op == "rotate":
        return _rotate(s["x"], s["table"][s["positions"]], case["interleaved"], case["backward"])
    if op == "append":
        return _append(s)
    if op == "weigh":
        return _weigh(s)
    return _evict(s)


# ------------------------------------------------------------------ the definition in 64 bits

def _wide(codes, params, bits):
    """fp64 values of packed rows."""
    c = codes.to(torch.int32)
    if bits == 4:
        c = torch.cat([(c % 16).unsqueeze(-1), (c // 16).unsqueeze(-1)], -1).reshape(*c.shape[:-1], -1)
    p = params.double()
    return c.double() * p[..., 0:1] + p[..., 1:2]


def _turned(x, rows, interleaved, sign):
    """fp64 rows as complex numbers times e^(i angle)."""
    r = rows.shape[1]
    x = x.double().clone()
    turn = torch.complex(rows[:, : r // 2].double(), sign * rows[:, r // 2:].double())[:, None]
    if interleaved:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:2], r // 2, 2).contiguous()) * turn
        x[..., :r] = torch.view_as_real(z).reshape(*x.shape[:2], r)
    else:
        z = torch.complex(x[..., : r // 2], x[..., r // 2:r]) * turn
        x[..., : r // 2], x[..., r // 2:r] = z.real, z.imag
    return x


def _exact_rows(x, bits):
    """fp64 values that bf16 rows [tokens, heads, dim] are held as."""
    x = x.double()
    lo, hi = x.min(-1).values, x.max(-1).values
    r = (hi - lo) / torch.full_like(lo, 2 ** bits - 1)
    s16 = r.to(torch.bfloat16)  # to nearest; one step up where that fell below r
    s16 = torch.where(s16.double() < r, (s16.view(torch.int16) + 1).view(torch.bfloat16), s16).double()
    c = ((x - lo[..., None]) / s16[..., None]).round()
    return torch.where(s16[..., None] > 0, c.clamp(0, 2 ** bits - 1) * s16[..., None], 0.0) + lo[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "table":
        at = torch.arange(case["rows"], device=DEV) if case["range"] else s["positions"]
        z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(at.double(), s["freqs"]))
        return torch.cat([z.real, z.imag], 1)
    if op == "rotate":
        return _turned(s["x"], s["table"][s["positions"]], case["interleaved"], -1.0 if case["backward"] else 1.0)
    d, bits, page, heads = case["dim"], case["bits"], case["page"], case["heads"]
    if op == "append":
        hq = case["qheads"]
        x = _turned(s["qkv"][:, :hq + heads], s["table"][s["positions"]], case["interleaved"], 1.0)
        kv = [_exact_rows(x[:, hq:].to(torch.bfloat16), bits), _exact_rows(s["qkv"][:, hq + heads:], bits)]
        for t in kv:
            t[s["slots"] < 0] = 0.0
        return (x[:, :hq], *kv)
    lens, qs = _lengths(case)
    if op == "evict":
        kept = torch.full((len(lens), heads, case["budget"]), -1, dtype=torch.int32)
        keys, values = [], []
        for b, n in enumerate(lens):
            at = s["table"][b, : -(-n // page)].long()
            w = s["weights"][at].transpose(0, 1).reshape(heads, -1)[:, :n].double().cpu()
            pick = []
            for h in range(heads):
                if n <= case["budget"]:
                    mine = torch.arange(n)
                else:
                    middle = w[h, case["first"]:n - case["last"]]
                    order = torch.argsort(-middle, stable=True)[: case["budget"] - case["first"] - case["last"]]
                    mine = torch.cat([torch.arange(case["first"]), order + case["first"],
                                      torch.arange(n - case["last"], n)]).sort().values
                kept[b, h, : len(mine)] = mine.to(torch.int32)
                pick.append(mine.to(DEV))
            for kv, out in ((0, keys), (1, values)):
                x = _wide(s["codes"][at, kv].transpose(0, 1).reshape(heads, -1, d * bits // 8),
                          s["params"][at, kv].transpose(0, 1).reshape(heads, -1, 2), bits)
                out.append(torch.stack([x[h, pick[h]] for h in range(heads)], 1))
            for h in range(heads):
                old, t = pick[h], torch.arange(len(pick[h]), device=DEV)
                s["weights"][s["new_table"][b].long()[t // page], h, t % page] = s["weights"][at[old // page], h,
                                                                                              old % page]
        return (torch.tensor([min(n, case["budget"]) for n in lens], dtype=torch.int32), kept, s["weights"].double(),
                torch.cat(keys), torch.cat(values))
    hq, w = case["qheads"], case["window"]
    out = s["weights"].double()
    first = 0
    for b, (n, nq) in enumerate(zip(lens, qs)):
        at = s["table"][b, : -(-n // page)].long()
        j = torch.arange(n, device=DEV)
        p = torch.arange(n - nq, n, device=DEV)[:, None]
        hidden = j > p
        if w:
            hidden |= j <= p - w
        for h in range(heads):
            k = _wide(s["codes"][at, 0, h].reshape(-1, d * bits // 8)[:n], s["params"][at, 0, h].reshape(-1, 2)[:n],
                      bits)
            total = torch.zeros(n, dtype=torch.float64, device=DEV)
            for g in range(h * (hq // heads), (h + 1) * (hq // heads)):
                a = s["q"][first:first + nq, g].double() @ k.T / math.sqrt(d)
                total += torch.softmax(a.masked_fill(hidden, float("-inf")), -1).sum(0)
            if case["sum"]:
                total[: n - nq] += s["previous"][at, h].reshape(-1)[: n - nq].double()
            some = j[max(0, n - nq + 1 - w) if w else 0:]
            out[at[some // page], h, some % page] = total[some]
        first += nq
    return out
