"""Every form of attention over the quantized cache, for both widths and both
bit counts, held to the bounds of tests/kv_reference.py.

The kernel is chosen by max_q * G (query rows of a head group: up to 8, up to
32, more).  Within a kernel the form follows from the sizes: contexts of one
tile of 128 tokens are not cut (no workspace); few and short ones run as
clusters that join by themselves (no workspace, up to 32 rows); the rest is
cut between blocks and joined by a second kernel (workspace).  Each test says
through the workspace's size which one it means.

Besides the bounds, a whole output lies within 2.0e-3 of the 64-bit one in the
Frobenius norm: its rounding to bf16 is 1.5e-3 to 1.7e-3 rms of values whose
mantissas are spread, and weights, keys and values rounded to 11 bits add 2e-4
each to its square; weights rounded to 8 bits would make it 2.3e-3.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import capi
from oracle import kv_cache as oracle
from tests.kv_reference import attended, check
from tests.test_gpu_kv_cache import Problem

pytestmark = pytest.mark.gpu

BAR = 2.0e-3
# rows a block: (query heads, cache heads, query tokens of a sequence at most)
ROWS = {8: [(16, 4, 2), (28, 4, 1), (4, 4, 8)], 16: [(16, 4, 8), (28, 4, 4), (4, 4, 32)],
        256: [(16, 4, 50), (28, 4, 5), (4, 4, 140)]}


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    from int8_quantized_linear_gb300 import build
    build.build()
    capi.lib()
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    yield
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


def workspace(p, hq, h, nq):
    b, width = p.table.shape
    return capi.i8ql_kv_attention_workspace(b, p.q.shape[0], hq, h, p.d, p.bits, p.page, width, nq)


def problem(batch, most, hq, h, nq, d, bits, page, seed):
    """`batch` sequences of up to `most` tokens (the first of just as many), with up to nq query tokens (the first of just
    as many; at least one elsewhere)."""
    rng = np.random.default_rng(seed)
    lens = [most] + rng.integers(1, most + 1, batch - 1).tolist()
    nqs = [nq] + rng.integers(1, nq + 1, batch - 1).tolist()
    return Problem(lens, nqs, hq, h, d, bits, page, seed)


def run(p, window, max_q):
    # (a draft's max_q is given even where every sequence has one token: the kernel goes by it)
    return p.run(window=window, single=False, max_q=max_q)


@pytest.mark.parametrize("layout", range(3))
@pytest.mark.parametrize("rows", [8, 16, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_cut_and_joined(bits, d, rows, layout):
    hq, h, nq = ROWS[rows][layout]
    p = problem(40, 700, hq, h, nq, d, bits, 32, rows + layout)
    assert workspace(p, hq, h, nq) > 0
    for window in (0, 150):
        y = run(p, window, nq)
        check(p, y, window=window, bar=BAR)
        assert torch.equal(run(p, window, nq), y)


@pytest.mark.parametrize("layout", range(3))
@pytest.mark.parametrize("rows", [8, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_clusters(bits, d, rows, layout):
    hq, h, nq = ROWS[rows][layout]
    p = problem(4, 2500, hq, h, nq, d, bits, 16, rows + layout)
    assert workspace(p, hq, h, nq) == 0 and p.table.shape[1] * p.page > 128
    for window in (0, 300):
        y = run(p, window, nq)
        check(p, y, window=window, bar=BAR if y.numel() >= 4096 else None)
        assert torch.equal(run(p, window, nq), y)


@pytest.mark.parametrize("layout", range(3))
@pytest.mark.parametrize("rows", [8, 16, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_contexts_of_one_tile_are_not_cut(bits, d, rows, layout):
    hq, h, nq = ROWS[rows][layout]
    p = problem(30, 112, hq, h, nq, d, bits, 16, rows + layout)  # (the table has one page more than a context)
    assert p.table.shape[1] * p.page <= 128 and workspace(p, hq, h, nq) == 0
    for window in (0, 20):
        y = run(p, window, nq)
        check(p, y, window=window, bar=BAR)
        assert torch.equal(run(p, window, nq), y)


@pytest.mark.parametrize("rows,nq", [(8, 2), (16, 7), (256, 30)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_contexts_of_many_parts(bits, d, rows, nq):
    """One head over a long context: an item in more parts than the joining kernel has warps."""
    p = Problem([20011, 130], [nq, 1], 4, 1, d, bits, 128, rows)
    assert workspace(p, 4, 1, nq) > 0
    y = run(p, 0, nq)
    check(p, y)
    assert torch.equal(run(p, 0, nq), y)


def test_offsets_past_32_bits_in_every_kernel():
    """A cache of more than 2^32 bytes, written and attended over at its end."""
    page, h, d, n = 256, 16, 128, 300
    pages = (1 << 32) // (2 * h * page * d) + 40
    codes = torch.empty((pages, 2, h, page, d), dtype=torch.uint8, device="cuda")
    params = torch.empty((pages, 2, h, page, 2), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((n, h, d), generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 30]], dtype=torch.int32)
    j = torch.arange(n)
    slots = (table[0, j // page].long() * page + j % page).cuda()
    capi.kv_cache_store(k.cuda(), v.cuda(), slots, codes, params)
    cached = [np.stack(x) for x in zip(*(oracle.quantize(x.float().numpy(), 8) for x in (k, v)))]
    for nq in (1, 3, 6, 60):
        q = torch.randn((nq, 2 * h, d), generator=g).to(torch.bfloat16)
        y = capi.kv_cache_attention(q.cuda(), codes, params, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                                    q_offsets=torch.tensor([0, nq], dtype=torch.int32).cuda(), max_q=nq)
        o, bound = attended(q.double(), *cached, nq, 0, d ** -0.5, 2 * nq > 32, 128)
        assert ((y.double().cpu() - o).abs() <= bound).all()
        assert (y.double().cpu() - o).norm() <= BAR * o.norm()
