"""Workloads of the quantized key/value cache: writing it, reading it back, attending over it.

Each case is one pass through an operator at sizes of real serving.  The head
layout of most cases (32 query heads over 8 cache heads of 128 channels, and
16 over 16) is that of the models whose projections this package benchmarks;
the rest are generic.
"""

from __future__ import annotations

import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 32 sequences: each writes one token, read back at once (latency)
        {"name": "write_step_32", "op": "write", "tokens": 32, "heads": 8, "dim": 128, "bits": 4, "page": 64,
         "holes": False},
        # a long prompt's keys and values, sliced out of the fused qkv projection
        {"name": "write_prompt_8192", "op": "write", "tokens": 8192, "heads": 8, "dim": 128, "bits": 4, "page": 64,
         "holes": False},
        # an 8-bit cache written by a padded batch: a fifth of the tokens have no slot
        {"name": "write_padded_1777_8bit", "op": "write", "tokens": 1777, "heads": 16, "dim": 64, "bits": 8,
         "page": 16, "holes": True},
        # a shared prefix read back to bf16 (to be moved or attended elsewhere)
        {"name": "read_prefix_16384", "op": "read", "tokens": 16384, "heads": 8, "dim": 128, "bits": 4, "page": 64,
         "holes": False},
        # a short odd-length prefix of an 8-bit cache with narrow heads
        {"name": "read_odd_1001_8bit", "op": "read", "tokens": 1001, "heads": 16, "dim": 64, "bits": 8, "page": 32,
         "holes": True},
        # one user, one token, a short context: launch and latency
        {"name": "attend_1x517", "op": "attend", "batch": 1, "kv": 517, "nq": 1, "qheads": 32, "heads": 8,
         "dim": 128, "bits": 4, "page": 64, "window": 0, "ragged": False},
        # an ordinary decode batch of mixed lengths
        {"name": "attend_64x4096", "op": "attend", "batch": 64, "kv": 4096, "nq": 1, "qheads": 32, "heads": 8,
         "dim": 128, "bits": 4, "page": 64, "window": 0, "ragged": True},
        # the largest decode batch, full contexts
        {"name": "attend_128x16384", "op": "attend", "batch": 128, "kv": 16384, "nq": 1, "qheads": 32, "heads": 8,
         "dim": 128, "bits": 4, "page": 64, "window": 0, "ragged": False},
        # every query head with a cache head of its own, 8 bits, small pages
        {"name": "attend_24x2047_8bit", "op": "attend", "batch": 24, "kv": 2047, "nq": 1, "qheads": 16, "heads": 16,
         "dim": 128, "bits": 8, "page": 16, "window": 0, "ragged": True},
        # two very long contexts: little parallel work but the cache's length
        {"name": "attend_2x131072", "op": "attend", "batch": 2, "kv": 131072, "nq": 1, "qheads": 32, "heads": 8,
         "dim": 128, "bits": 4, "page": 128, "window": 0, "ragged": False},
        # checking up to five drafted tokens a sequence, sliding window, odd head group, narrow heads
        {"name": "attend_20x3001_draft", "op": "attend", "batch": 20, "kv": 3001, "nq": 5, "qheads": 28, "heads": 4,
         "dim": 64, "bits": 4, "page": 32, "window": 1024, "ragged": True},
        # prompt chunks attending over what is already cached and themselves
        {"name": "attend_prompt_2x2048", "op": "attend", "batch": 2, "kv": 8192, "nq": 2048, "qheads": 32,
         "heads": 8, "dim": 128, "bits": 4, "page": 64, "window": 0, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    dim, bits, page = rng.choice([64, 128, 128]), rng.choice([4, 4, 8]), rng.choice([16, 32, 64, 128, 256])
    if kind != "attend":
        heads = rng.choice([1, 2, 3, 4, 5, 8, 16])
        most = (8192 if kind == "write" else 16384) * 8 * 128 // (heads * dim)
        return {"op": kind, "tokens": _log(rng, 16, min(most, 16384)), "heads": heads, "dim": dim, "bits": bits,
                "page": page, "holes": rng.random() < 0.5}
    heads, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if rng.random() < 0.6:  # single tokens or a few drafted ones
        nq = rng.choice([1, 1, 1, 2, 4, 7])
        batch = _log(rng, 1, 128)
        kv = _log(rng, max(nq, 100), min(131072, max(256, 128 * 16384 * 8 // (2 * batch * heads * group))))
    else:  # prompts
        nq = _log(rng, 16, 2048)
        batch = _log(rng, 1, 8)
        kv = nq + _log(rng, 1, 6144)
        while batch * nq * kv * heads * group > 2 * 2048 * 8192 * 32:
            batch, nq = max(1, batch // 2), max(16, nq // 2)
    return {"op": "attend", "batch": batch, "kv": kv, "nq": nq, "qheads": heads * group, "heads": heads, "dim": dim,
            "bits": bits, "page": page, "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
            "ragged": rng.random() < 0.6}


def _lengths(case):
    """Cache length and query tokens of each sequence: part of the case, the same for every seed."""
    b, kv, nq = case["batch"], case["kv"], case["nq"]
    if not case["ragged"]:
        return [kv] * b, [nq] * b
    r = random.Random("%d %d %d" % (b, kv, nq))
    lens = [kv] + [r.randint(1, kv) for _ in range(b - 1)]
    qs = [nq] + [r.randint(1, nq) for _ in range(b - 1)]
    return lens, [min(q, n) for q, n in zip(qs, lens)]


def _row_bytes(case):
    return case["dim"] * case["bits"] // 8 + 4  # codes, scale and low value of one token of one head


def work(case):
    if case["op"] in ("write", "read"):
        t, h, d = case["tokens"], case["heads"], case["dim"]
        full, packed = 2 * t * h * d * 2, 2 * t * h * _row_bytes(case)
        if case["op"] == "read":
            return {"bytes": packed + full + 8 * t, "flops": 2 * full}
        # written, then read back: the inputs, the cache out and in, the values out
        return {"bytes": 2 * full + 2 * packed + 16 * t, "flops": 6 * full}
    lens, qs = _lengths(case)
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
    rows = sum(qs) * case["qheads"] * case["dim"]
    return {"bytes": 2 * seen * case["heads"] * _row_bytes(case) + 4 * rows + 4 * seen // case["page"],
            "flops": 4 * pairs * case["qheads"] * case["dim"]}


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


def prepare(case, seed):
    g = _gen(seed)
    d, bits, page, heads = case["dim"], case["bits"], case["page"], case["heads"]
    if case["op"] in ("write", "read"):
        t = case["tokens"]
        pages = -(-t // page) + 3
        order = torch.randperm(pages, generator=g, device=DEV)[: -(-t // page)]
        slots = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:t].contiguous()
        if case["holes"]:
            slots[torch.rand(t, generator=g, device=DEV) < 0.2] = -1
        codes = torch.randint(0, 256, (pages, 2, heads, page, d * bits // 8), generator=g, device=DEV,
                              dtype=torch.uint8)
        params = torch.rand((pages, 2, heads, page, 2), generator=g, device=DEV)
        params[..., 1] = -params[..., 1] * (2 ** bits - 1) / 2
        s = {"case": case, "slots": slots, "codes": codes, "params": params.to(torch.bfloat16)}
        if case["op"] == "write":
            # keys and values as slices of a fused projection's rows: 4 query heads beside each cache head
            qkv = torch.cat([torch.empty((t, 4 * heads, d), device=DEV, dtype=torch.bfloat16).zero_(),
                             _heads(g, t, heads, d, 8.0), _heads(g, t, heads, d, 1.0)], dim=1)
            s["k"], s["v"] = qkv[:, 4 * heads:5 * heads], qkv[:, 5 * heads:]
        return s
    lens, qs = _lengths(case)
    b, wide = case["batch"], -(-max(lens) // page)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    table = torch.full((b, wide), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = table.to(DEV)
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
    codes = torch.empty((pages, 2, heads, page, d * bits // 8), dtype=torch.uint8, device=DEV)
    params = torch.empty((pages, 2, heads, page, 2), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 28) // (heads * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        for kv in (0, 1):
            x = _heads(g, n * page, heads, d, 1.0 if kv else 4.0).view(n, page, heads, d).transpose(1, 2)
            c, p = _quantize(x.float(), bits)
            codes[i:i + n, kv] = _pack(c, bits)
            params[i:i + n, kv] = p
    # what lies behind a sequence's end in its last page was never written
    for i, n in enumerate(lens):
        if n % page:
            params[order[sum(need[:i + 1]) - 1].long(), :, :, n % page:] = float("nan")
    q = _heads(g, sum(qs), case["qheads"], d, 1.0)
    offsets = torch.zeros(b + 1, dtype=torch.int32)
    offsets[1:] = torch.tensor(qs, dtype=torch.int32).cumsum(0)
    return {"case": case, "q": q, "codes": codes, "params": params, "table": table,
            "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "offsets": offsets.to(DEV), "max_q": max(qs)}


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


def _write(s):
    page, bits = s["case"]["page"], s["case"]["bits"]
    there = s["slots"] >= 0
    at = s["slots"][there]
    x = torch.stack([s["k"], s["v"]], 1)[there].float()
    c, p = _quantize(x, bits)
    s["codes"][at // page, :, :, at % page] = _pack(c, bits)
    s["params"][at // page, :, :, at % page] = p


def _attend(s):
    case = s["case"]
    b, hq, h, d, page = case["batch"], case["qheads"], case["heads"], case["dim"], case["page"]
    mq, wide = s["max_q"], s["table"].shape[1]
    at = s["table"].clamp(min=0).long()
    lens = s["lens"].long()
    nq = (s["offsets"][1:] - s["offsets"][:-1]).long()
    j = torch.arange(wide * page, device=DEV)
    live = (j < lens[:, None])[:, None, :, None]
    # [batch, pages, K/V, heads, page, .] -> [batch, heads, tokens, .]
    flat = lambda x, kv: x[at, kv].transpose(1, 2).flatten(2, 3)  # noqa: E731
    k, v = (_values(flat(s["codes"], kv), torch.where(live, flat(s["params"], kv), torch.zeros((), device=DEV,
                    dtype=torch.bfloat16)), case["bits"]) for kv in (0, 1))
    i = torch.arange(mq, device=DEV)
    row = (s["offsets"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)  # [batch, max_q]
    q = s["q"].float()[row].view(b, mq, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, hq // h * mq, d)
    pos = (lens - nq)[:, None] + i  # [batch, max_q]
    see = j <= pos[..., None]
    if case["window"]:
        see &= j > pos[..., None] - case["window"]
    x = torch.matmul(q, k.transpose(2, 3)).view(b, h, hq // h, mq, -1) * d ** -0.5
    x = torch.where(see[:, None, None], x, torch.full((), float("-inf"), device=DEV))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, h, hq // h * mq, -1), v).view(b, h, hq // h, mq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(b, mq, hq, d)
    return o[i < nq[:, None]].to(torch.bfloat16)


def run(state):
    case, s = state["case"], state
    if own:
        from int8_quantized_linear_gb300 import capi
        if case["op"] == "write":
            capi.kv_cache_store(s["k"], s["v"], s["slots"], s["codes"], s["params"])
        if case["op"] in ("write", "read"):
            return capi.kv_cache_load(s["codes"], s["params"], s["slots"], case["dim"])
        if case["nq"] == 1:
            return capi.kv_cache_attention(s["q"], s["codes"], s["params"], s["table"], s["lens"],
                                           window=case["window"])
        return capi.kv_cache_attention(s["q"], s["codes"], s["params"], s["table"], s["lens"],
                                       q_offsets=s["offsets"], max_q=s["max_q"], window=case["window"])
    if case["op"] == "write":
        _write(s)
    if case["op"] in ("write", "read"):
        return _read(s)
    return _attend(s)


# ------------------------------------------------------------------ the definition in 64 bits

def _wide(codes, params, bits):
    """fp64 values of packed rows."""
    c = codes.to(torch.int32)
    if bits == 4:
        c = torch.cat([(c % 16).unsqueeze(-1), (c // 16).unsqueeze(-1)], -1).reshape(*c.shape[:-1], -1)
    p = params.double()
    return c.double() * p[..., 0:1] + p[..., 1:2]


def exact(case, seed):
    s = prepare(case, seed)
    d, bits, page, heads = case["dim"], case["bits"], case["page"], case["heads"]
    if case["op"] in ("write", "read"):
        out = []
        for kv in (0, 1):
            if case["op"] == "write":
                x = (s["v"] if kv else s["k"]).double()
                lo, hi = x.min(-1).values, x.max(-1).values
                r = (hi - lo) / torch.full_like(lo, 2 ** bits - 1)
                s16 = r.to(torch.bfloat16)  # to nearest; one step up where that fell below r
                s16 = torch.where(s16.double() < r, (s16.view(torch.int16) + 1).view(torch.bfloat16), s16).double()
                c = ((x - lo[..., None]) / s16[..., None]).round()
                x = torch.where(s16[..., None] > 0, c.clamp(0, 2 ** bits - 1) * s16[..., None], 0.0) + lo[..., None]
            else:
                at = s["slots"].clamp(min=0)
                page_of = s["codes"][:, kv].transpose(1, 2).reshape(-1, heads, d * bits // 8)
                param_of = s["params"][:, kv].transpose(1, 2).reshape(-1, heads, 2)
                x = _wide(page_of[at], param_of[at], bits)
            x[s["slots"] < 0] = 0.0
            out.append(x)
        return tuple(out)
    lens, qs = _lengths(case)
    hq, w = case["qheads"], case["window"]
    rows, first = [], 0
    for b, (n, nq) in enumerate(zip(lens, qs)):
        at = s["table"][b, : -(-n // page)].long()
        j = torch.arange(n, device=DEV)
        p = torch.arange(n - nq, n, device=DEV)[:, None]
        hidden = j > p
        if w:
            hidden |= j <= p - w
        o = torch.empty((nq, hq, d), dtype=torch.float64, device=DEV)
        for h in range(heads):
            k, v = (_wide(s["codes"][at, kv, h].reshape(-1, d * bits // 8)[:n], s["params"][at, kv, h].reshape(-1, 2)[:n],
                          bits) for kv in (0, 1))
            g = slice(h * (hq // heads), (h + 1) * (hq // heads))
            q = s["q"][first:first + nq, g].double()
            a = torch.einsum("qgd,kd->gqk", q, k) / d ** 0.5
            a = torch.softmax(a.masked_fill(hidden, float("-inf")), -1)
            o[:, g] = torch.einsum("gqk,kd->qgd", a, v)
        rows.append(o)
        first += nq
    return torch.cat(rows)
