"""An attention block of a served model on the quantized key/value cache.

int8 weight-only projections (``w8a16_gemm``), keys and values quantized into
a paged 4- or 8-bit cache as the fused projection produces them
(``kv_cache_store``, straight from its rows), attention over the cache
(``kv_cache_attention``) for prompt chunks and single tokens in one batch, and
the output projection.  Rotary or other position encodings are the caller's:
they act on the q and k slices between the projection and the store.

    python examples/attention_block.py

runs a prompt of two sequences and a few decode steps, reads the cache back
(``kv_cache_load``) and compares with plain attention over what it reads.
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
                 device="cuda"):
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

    def forward(self, x, batch):
        """x bf16 [tokens, hidden]: the new tokens of the sequences in `batch`
        (pairs of a sequence's name and its number of new tokens), in order.
        Returns bf16 [tokens, hidden]."""
        slots, table = [], torch.zeros((len(batch), self.width), dtype=torch.int32)
        for i, (name, n) in enumerate(batch):
            mine = self.pages.setdefault(name, [])
            begin = self.lengths.get(name, 0)
            while len(mine) * self.page_size < begin + n:
                mine.append(self.free.pop())
            slots += [mine[t // self.page_size] * self.page_size + t % self.page_size for t in range(begin, begin + n)]
            self.lengths[name] = begin + n
            table[i, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
        counts = torch.tensor([0] + [n for _, n in batch], dtype=torch.int32)
        offsets = counts.cumsum(0).to(torch.int32)
        lens = torch.tensor([self.lengths[name] for name, _ in batch], dtype=torch.int32)
        slots, table, offsets, lens = (t.to(self.device, non_blocking=True)
                                       for t in (torch.tensor(slots, dtype=torch.int64), table, offsets, lens))

        rows = capi.w8a16_gemm(x, *self.qkv).view(x.shape[0], self.q_heads + 2 * self.heads, self.head_dim)
        q, k, v = rows.split([self.q_heads, self.heads, self.heads], dim=1)
        capi.kv_cache_store(k, v, slots, self.codes, self.params)
        out = capi.kv_cache_attention(q, self.codes, self.params, table, lens, q_offsets=offsets,
                                      max_q=max(n for _, n in batch))
        self.last_q = q
        return capi.w8a16_gemm(out.view(x.shape[0], -1), *self.o), out

    def read(self, name):
        """The sequence's keys and values, bf16 [length, heads, head_dim]."""
        n, mine = self.lengths[name], self.pages[name]
        slots = torch.tensor([mine[t // self.page_size] * self.page_size + t % self.page_size for t in range(n)],
                             dtype=torch.int64, device=self.device)
        return capi.kv_cache_load(self.codes, self.params, slots, self.head_dim)

    def release(self, name):
        self.free += self.pages.pop(name)
        del self.lengths[name]


def plain_attention(q, k, v):
    """fp64 causal attention of the last len(q) tokens over k and v."""
    q, k, v = q.double(), k.double(), v.double()
    n, nq, group = k.shape[0], q.shape[0], q.shape[1] // k.shape[1]
    x = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(group, 1)) * q.shape[2] ** -0.5
    hidden = torch.arange(n, device=q.device) > torch.arange(n - nq, n, device=q.device)[:, None]
    return torch.einsum("hqk,khd->qhd", torch.softmax(x.masked_fill(hidden, float("-inf")), -1),
                        v.repeat_interleave(group, 1))


def main(hidden=2560, q_heads=32, heads=8, head_dim=128, bits=4, prompts=(300, 77), steps=5):
    """Worst relative error of an attention output over the run."""
    block = AttentionBlock(hidden, q_heads, heads, head_dim, bits=bits)
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
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    for name in names:
        block.release(name)
    return worst


if __name__ == "__main__":
    for bits in (4, 8):
        print(f"{bits}-bit cache: attention over it within {main(bits=bits):.2e} of plain attention over its values")
