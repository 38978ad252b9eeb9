"""An attention block of a served model on the quantized key/value cache.

int8 weight-only projections (``w8a16_gemm``), keys and values quantized into
a paged 4- or 8-bit cache as the fused projection produces them
(``kv_cache_store``, straight from its rows), attention over the cache
(``kv_cache_attention``) for prompt chunks and single tokens in one batch, and
the output projection.  With ``rotary`` the queries and keys are turned by their
positions as they are stored (``kv_cache_store_rotary``, from a table made by
``rotary_table``); other position encodings are the caller's: they act on the q
and k slices between the projection and the store.  With ``budget`` a sequence
keeps at most that many tokens: the block sums up how much attention each gets
(``kv_cache_weights``) and after a step that left more drops those that got least
(``kv_cache_evict``).

    python examples/attention_block.py

runs a prompt of two sequences and a few decode steps, reads the cache back
(``kv_cache_load``) and compares with plain attention over what it reads; then
the same with rotary positions and contexts cut to a budget.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from int8_quantized_linear_gb300 import capi  # noqa: E402


class AttentionBlock:
    """Projections, a pool of cache pages, and the sequences living in it."""

    def __init__(self, hidden, q_heads, heads, head_dim, *, bits=4, pages=64, page_size=64, max_tokens=4096, seed=0,
                 rotary=None, budget=None, recent=16, device="cuda"):
        """max_tokens: the most that a sequence holds at a time.  rotary: frequencies (``rotary_frequencies``) of the
        rotary channels, or None.  budget: tokens a sequence keeps, its first 4 and its last `recent` among them, or
        None."""
        if budget is not None and not 0 <= recent <= budget:
            raise ValueError(f"the last {recent} tokens are not a part of a budget of {budget}")
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.q_heads, self.heads, self.head_dim, self.page_size = q_heads, heads, head_dim, page_size
        width = (q_heads + 2 * heads) * head_dim

        def weight(n, k):
            w = (torch.randn((n, k), generator=g, device=device) * k ** -0.5).to(torch.bfloat16)
            return capi.quantize_weight_per_channel_int8(w)

        self.qkv, self.o = weight(width, hidden), weight(hidden, q_heads * head_dim)
        self.codes, self.params = capi.kv_cache_alloc(pages, heads, page_size, head_dim, bits, device)
        self.free = list(range(pages))
        self.pages, self.lengths = {}, {}  # per sequence
        self.width = -(-max_tokens // page_size)
        self.device = device
        self.positions = {}  # of a sequence's next token; they go on where its length is cut
        self.rotary = rotary
        self.table = None if rotary is None else capi.rotary_table(rotary, max_tokens)
        self.budget, self.recent = budget, recent
        self.weights = None if budget is None else torch.zeros((pages, heads, page_size), device=device)

    def forward(self, x, batch):
        """x bf16 [tokens, hidden]: the new tokens of the sequences in `batch`
        (pairs of a sequence's name and its number of new tokens), in order.
        Returns bf16 [tokens, hidden]."""
        end = max((self.positions.get(name, 0) + n for name, n in batch), default=0)
        if self.table is not None and end > self.table.shape[0]:
            self.table = capi.rotary_table(self.rotary, max(end, 2 * self.table.shape[0]))
        slots, places, table = [], [], torch.zeros((len(batch), self.width), dtype=torch.int32)
        for i, (name, n) in enumerate(batch):
            mine = self.pages.setdefault(name, [])
            begin = self.lengths.get(name, 0)
            while len(mine) * self.page_size < begin + n:
                mine.append(self.free.pop())
            slots += [mine[t // self.page_size] * self.page_size + t % self.page_size for t in range(begin, begin + n)]
            self.lengths[name] = begin + n
            at = self.positions.get(name, 0)
            places += range(at, at + n)
            self.positions[name] = at + n
            table[i, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
        counts = torch.tensor([0] + [n for _, n in batch], dtype=torch.int32)
        offsets = counts.cumsum(0).to(torch.int32)
        lens = torch.tensor([self.lengths[name] for name, _ in batch], dtype=torch.int32)
        slots, places, table, offsets, lens = (
            t.to(self.device, non_blocking=True)
            for t in (torch.tensor(slots, dtype=torch.int64), torch.tensor(places, dtype=torch.int64), table, offsets, lens))

        rows = capi.w8a16_gemm(x, *self.qkv).view(x.shape[0], self.q_heads + 2 * self.heads, self.head_dim)
        q, k, v = rows.split([self.q_heads, self.heads, self.heads], dim=1)
        if self.table is None:
            capi.kv_cache_store(k, v, slots, self.codes, self.params)
        else:
            q = capi.kv_cache_store_rotary(q, k, v, self.table, slots, self.codes, self.params, positions=places)
        max_q = max(n for _, n in batch)
        out = capi.kv_cache_attention(q, self.codes, self.params, table, lens, q_offsets=offsets, max_q=max_q)
        self.last_q = q
        if self.budget is not None:
            capi.kv_cache_weights(q, self.codes, self.params, table, lens, self.weights, q_offsets=offsets, max_q=max_q,
                                  previous=self.weights)
        return capi.w8a16_gemm(out.view(x.shape[0], -1), *self.o), out

    def read(self, name):
        """The sequence's keys and values, bf16 [length, heads, head_dim]."""
        n, mine = self.lengths[name], self.pages[name]
        slots = torch.tensor([mine[t // self.page_size] * self.page_size + t % self.page_size for t in range(n)],
                             dtype=torch.int64, device=self.device)
        return capi.kv_cache_load(self.codes, self.params, slots, self.head_dim)

    def cut(self, names):
        """Brings the sequences down to the budget, and gives back the pages that they then no longer need."""
        names = [n for n in names if self.lengths[n] > self.budget]
        if not names:
            return
        table = torch.zeros((len(names), self.width), dtype=torch.int32)
        for i, name in enumerate(names):
            table[i, :len(self.pages[name])] = torch.tensor(self.pages[name], dtype=torch.int32)
        lens = torch.tensor([self.lengths[n] for n in names], dtype=torch.int32)
        capi.kv_cache_evict(self.codes, self.params, self.weights, table.to(self.device), lens.to(self.device), self.budget,
                            first=min(4, self.budget - self.recent), last=self.recent)
        for name in names:
            self.lengths[name] = self.budget
            keep = -(-self.budget // self.page_size)
            self.free += self.pages[name][keep:]
            self.pages[name] = self.pages[name][:keep]

    def release(self, name):
        self.free += self.pages.pop(name)
        del self.lengths[name], self.positions[name]


def plain_attention(q, k, v):
    """fp64 causal attention of the last len(q) tokens over k and v."""
    q, k, v = q.double(), k.double(), v.double()
    n, nq, group = k.shape[0], q.shape[0], q.shape[1] // k.shape[1]
    x = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(group, 1)) * q.shape[2] ** -0.5
    hidden = torch.arange(n, device=q.device) > torch.arange(n - nq, n, device=q.device)[:, None]
    return torch.einsum("hqk,khd->qhd", torch.softmax(x.masked_fill(hidden, float("-inf")), -1),
                        v.repeat_interleave(group, 1))


def main(hidden=2560, q_heads=32, heads=8, head_dim=128, bits=4, prompts=(300, 77), steps=5, rotary=None, budget=None):
    """Worst relative error of an attention output over the run."""
    block = AttentionBlock(hidden, q_heads, heads, head_dim, bits=bits, rotary=rotary, budget=budget)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    worst = 0.0
    names = [f"sequence {i}" for i in range(len(prompts))]
    for step in range(steps + 1):
        batch = list(zip(names, prompts)) if step == 0 else [(n, 1) for n in names]
        x = torch.randn((sum(n for _, n in batch), hidden), generator=g, device="cuda").to(torch.bfloat16)
        y, out = block.forward(x, batch)
        assert y.shape == x.shape and bool(torch.isfinite(y.float()).all())
        at = 0
        for name, n in batch:
            k, v = block.read(name)
            ref = plain_attention(block.last_q[at:at + n], k, v)
            worst = max(worst, float((out[at:at + n].double() - ref).norm() / ref.norm()))
            at += n
        if budget is not None:
            block.cut(names)
            assert all(block.lengths[n] <= budget for n in names)
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    for name in names:
        block.release(name)
    return worst


if __name__ == "__main__":
    for bits in (4, 8):
        print(f"{bits}-bit cache: attention over it within {main(bits=bits):.2e} of plain attention over its values")
        far = main(bits=bits, rotary=capi.rotary_frequencies(128, 1e6), budget=128)
        print(f"  with rotary positions, contexts cut to 128 tokens: {far:.2e}")
