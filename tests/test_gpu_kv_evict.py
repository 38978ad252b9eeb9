"""GPU tests of cache eviction through the binding: attention weights summed per
token within bounds of fp32 arithmetic (oracle/kv_evict.py), the kept tokens and
what moves with them exactly, and both together with rotary positions and
attention, as a serving loop uses them."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import capi
from oracle import kv_cache as cache_oracle
from oracle import kv_evict as oracle
from tests import kv_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    from int8_quantized_linear_gb300 import build
    build.build()
    capi.lib()
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    yield
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


class Cache:
    """Sequences of random keys in pages that lie anywhere; what belongs to no token is NaN."""

    def __init__(self, lens, hq, heads, d, bits, page, nqs=None, seed=0, spread=1.0, wide=0, spare=2):
        rng = np.random.default_rng(seed)
        self.lens, self.nqs = list(lens), list(nqs or [1] * len(lens))
        self.page, self.bits, self.d, self.heads = page, bits, d, heads
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max([*need, 1]) + wide), -7, np.int32)  # (not a page)
        codes = np.full((self.pages, 2, heads, page, d), 3, np.uint8)
        params = np.full((self.pages, 2, heads, page, 2), np.nan, np.float32)
        self.seqs, at = [], 0
        for i, n in enumerate(lens):
            self.table[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
            x = rng.standard_normal((n, heads, d)).astype(np.float32) * spread
            x[..., rng.integers(0, d)] *= 5
            x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
            c, s, low = cache_oracle.quantize(x, bits) if n else (np.zeros((0, heads, d), np.uint8),) + 2 * (np.zeros((0, heads)),)
            self.seqs.append((c, s, low))
            j = np.arange(n)
            pages, off = self.table[i, j // page], j % page
            codes[pages, 0, :, off] = c
            params[pages, 0, :, off] = np.stack([s, low], -1)
            codes[pages, 1, :, off] = rng.integers(0, 2 ** bits, c.shape)
            params[pages, 1, :, off] = rng.standard_normal((n, heads, 2))
        self.codes = torch.from_numpy(cache_oracle.pack(codes, bits)).cuda()
        self.params = torch.from_numpy(params).to(torch.bfloat16).cuda()
        self.q = torch.from_numpy(rng.standard_normal((sum(self.nqs), hq, d)).astype(np.float32)).to(torch.bfloat16)
        self.previous = rng.random((self.pages, heads, page)).astype(np.float32)
        self.rng = rng

    def gpu(self):
        offsets = torch.tensor([0, *self.nqs], dtype=torch.int32).cumsum(0).to(torch.int32)
        return {"codes": self.codes, "params": self.params, "page_table": torch.from_numpy(self.table).cuda(),
                "kv_lens": torch.tensor(self.lens, dtype=torch.int32).cuda()}, offsets.cuda()

    def weigh(self, window=0, scale=None, previous=None, weights=None, q=None, max_q=None, offsets=True, **more):
        args, at = self.gpu()
        weights = torch.full((self.pages, self.heads, self.page), -5.0, device="cuda") if weights is None else weights
        if offsets:
            more.update(q_offsets=at, max_q=max(self.nqs) if max_q is None else max_q)
        got = capi.kv_cache_weights(self.q.cuda() if q is None else q, weights=weights, window=window, scale=scale,
                                    previous=previous, **args, **more)
        assert got.data_ptr() == weights.data_ptr()
        return got

    def check(self, got, window=0, scale=None, previous=None):
        """Every weight within its bound; what no query sees as it was (-5)."""
        got = got.cpu().numpy().astype(np.float64)
        want, bound = np.full(got.shape, -5.0), np.zeros(got.shape)
        at = 0
        for i, (n, nq) in enumerate(zip(self.lens, self.nqs)):
            q = self.q[at:at + nq].double().numpy()
            at += nq
            w, b, seen = oracle.weights(q, *self.seqs[i], nq, window, self.d ** -0.5 if scale is None else scale,
                                        2 ** (self.bits - 1))
            j = np.arange(n)[seen]
            pages, off = self.table[i, j // self.page], j % self.page
            if previous is not None:
                w = w + np.where(np.arange(n) < n - nq, previous_of(previous, self.table[i], n, self.page), 0.0)
                b = b + 2.0 ** -23 * np.abs(w)
            want[pages, :, off], bound[pages, :, off] = w.T[seen], b.T[seen]
        off = np.abs(got - want)
        assert (off <= bound).all(), f"off by {np.nanmax(off / np.maximum(bound, 1e-300)):.3g} of the bound"


def previous_of(previous, pages, n, page):
    j = np.arange(n)
    return previous[pages[j // page], :, j % page].T.astype(np.float64) if n else np.zeros((previous.shape[1], 0))


FEW = [  # lens, nqs, hq, heads, page, window
    ([1], [1], 1, 1, 16, 0),
    ([517], [1], 32, 8, 64, 0),
    ([300, 1, 77, 129], [1, 1, 1, 1], 12, 4, 32, 0),
    ([64, 700, 0, 33], [3, 7, 0, 5], 8, 2, 16, 0),
    ([5, 2, 0, 400], [6, 2, 2, 1], 5, 5, 128, 0),      # more queries than tokens: rows that see nothing
    ([1000, 90], [2, 2], 16, 1, 256, 70),
    ([333, 2000], [4, 4], 14, 2, 64, 1),
    ([129] * 40, [1] * 40, 6, 3, 16, 0),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(FEW)))
def test_weights_few_rows(case, d, bits):
    lens, nqs, hq, heads, page, window = FEW[case]
    c = Cache(lens, hq, heads, d, bits, page, nqs, seed=case + d + bits)
    c.check(c.weigh(window), window)
    previous = torch.from_numpy(c.previous).cuda()
    c.check(c.weigh(window, previous=previous), window, previous=c.previous)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,nqs,hq,heads,page,window", [
    ([1], [40], 1, 1, 16, 0),                               # one row of forty sees anything
    ([300], [33], 2, 2, 32, 0),
    ([257, 128, 640], [64, 128, 3], 4, 2, 64, 0),
    ([900, 20, 0, 470], [129, 20, 0, 1], 8, 2, 16, 0),
    ([500, 260], [257, 260], 7, 7, 128, 0),
    ([700, 333], [90, 50], 12, 3, 256, 100),
    ([1500], [600], 3, 1, 64, 33),
])
def test_weights_many_rows(lens, nqs, hq, heads, page, window, d, bits):
    c = Cache(lens, hq, heads, d, bits, page, nqs, seed=d + bits + len(lens))
    c.check(c.weigh(window), window)
    previous = torch.from_numpy(c.previous).cuda()
    c.check(c.weigh(window, previous=previous), window, previous=c.previous)


@pytest.mark.parametrize("hq,nq", [(4, 670), (4, 1030), (1, 2600)])
def test_weights_row_blocks_in_groups(hq, nq):
    """A table so wide that several row blocks share a sum (the last of them with and without a second half)."""
    c = Cache([nq + 300, 40], hq, 1, 64, 4, 256, [nq, 33], seed=nq, wide=(1 << 20) // 256)
    c.check(c.weigh())


@pytest.mark.parametrize("nqs", [[1, 1], [50, 40]])
def test_weights_scales_and_magnitudes(nqs):
    for scale, spread in ((-0.2, 1.0), (0.0, 1.0), (30.0, 1.0), (1e-3, 1e4), (0.05, 1e-20), (1e-30, 1e28)):
        c = Cache([400, 131], 4, 2, 128, 4, 32, nqs, seed=7, spread=spread)
        got = c.weigh(scale=scale)
        c.check(got, scale=scale)


@pytest.mark.parametrize("nqs", [[1, 1, 1], [3, 2, 4], [100, 60, 70]])
def test_weights_sum_to_the_rows(nqs):
    """Each row's weights sum to 1, so a head's to its rows (fp32 sums of n terms: n 2^-24 and the exponentials' 2^-20)."""
    c = Cache([4000, 250, 1111], 8, 2, 128, 8, 64, nqs, seed=5)
    w = c.weigh(weights=torch.zeros((c.pages, 2, 64), device="cuda")).cpu().double()
    for i, nq in enumerate(nqs):
        total = w[torch.from_numpy(c.table[i][c.table[i] >= 0]).long()].sum((0, 2))
        assert ((total - 4 * nq).abs() <= 4 * nq * (2.0 ** -20 + 4500 * 2.0 ** -24)).all()


@pytest.mark.parametrize("nqs", [[1, 2], [40, 70]])
def test_weights_in_place_queries_sliced_and_repeatable(nqs):
    c = Cache([500, 333], 6, 3, 64, 4, 16, nqs, seed=3)
    fresh = c.weigh()
    qkv = torch.full((sum(nqs), 12, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:, 2:8] = c.q.cuda()
    again = c.weigh(q=qkv[:, 2:8])
    assert torch.equal(fresh, again)
    previous = torch.from_numpy(c.previous).cuda()
    other = c.weigh(previous=previous)
    both = previous.clone()
    c.weigh(previous=both, weights=both)
    seen = other != -5.0
    assert torch.equal(other[seen], both[seen]) and torch.equal(both[~seen], previous[~seen])
    # a larger bound of the queries: another kernel perhaps, the same sums within the bounds
    c.check(c.weigh(max_q=sum(nqs)))


def test_weights_not_finite_where_unseen():
    """Rows behind the end and before the window may hold anything."""
    for nqs in ([1, 1], [45, 20]):
        c = Cache([300, 90], 4, 2, 64, 8, 16, nqs, seed=2)
        args, _ = c.gpu()
        window = 25
        for i, n in enumerate(c.lens):
            first = n - nqs[i] + 1 - window
            for j in range(0, first):
                c.params[c.table[i, j // 16], :, :, j % 16] = float("inf")
        c.check(c.weigh(window), window)
        # pages that nothing sees any more may be anybody's
        c.table[0, : (300 - nqs[0] + 1 - window) // 16] = -1
        c.check(c.weigh(window), window)
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


@pytest.mark.parametrize("nqs", [[1, 1], [45, 20]])
def test_weights_bad_input_is_recorded(nqs):
    def fresh():
        return Cache([300, 90], 4, 2, 64, 8, 16, nqs, seed=2)
    c = fresh()
    for bad in (-1, c.pages, 1 << 30):
        c = fresh()
        c.table[1, 2] = bad
        got = c.weigh()
        assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX
        # sequence 0 is as it should be, and no weight has gone where it should not
        c.lens[1] = c.nqs[1] = 0
        keep = torch.ones(c.pages, dtype=torch.bool)
        keep[torch.from_numpy(c.table[1][(c.table[1] >= 0) & (c.table[1] < c.pages)]).long()] = False
        want = c.q
        c.q = c.q[: nqs[0]]
        c.nqs = [nqs[0], 0]
        ref = c.weigh()
        assert torch.equal(got[keep], ref[keep])
        c.q = want
    c = fresh()
    c.lens[1] = 1 << 28
    c.weigh()
    assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX
    if nqs[0] > 1:
        c = fresh()
        c.weigh(max_q=nqs[0] - 1)
        assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX


def test_weights_nothing_to_do():
    c = Cache([30, 20], 4, 2, 64, 4, 16, [0, 0])
    got = c.weigh(max_q=5)
    assert (got == -5.0).all()


def test_binding_refusals():
    codes, params = capi.kv_cache_alloc(6, 2, 16, 64)
    w = torch.zeros((6, 2, 16), device="cuda")
    table, lens = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    ok = {"q": q, "codes": codes, "params": params, "page_table": table, "kv_lens": lens, "weights": w}
    for name, bad in (("weights", w[:5]), ("previous", w[:5]), ("kv_lens", lens[:1]), ("page_table", lens), ("q", q[0]),
                      ("weights", w.cpu()), ("previous", w.cpu()), ("weights", w.transpose(1, 2))):
        with pytest.raises(ValueError, match=name):
            capi.kv_cache_weights(**{**ok, name: bad})
    for name, bad in (("weights", w.double()), ("previous", w.half()), ("q", q.float()), ("kv_lens", lens.long())):
        with pytest.raises(TypeError, match=name):
            capi.kv_cache_weights(**{**ok, name: bad})
    small = torch.empty(15, dtype=torch.uint8, device="cuda")
    many = {**ok, "q": torch.zeros((40, 4, 64), dtype=torch.bfloat16, device="cuda")}
    with pytest.raises(capi.I8qlError):
        capi.kv_cache_weights(**many, q_offsets=torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda"), max_q=20,
                              workspace=small)
    ok = {"codes": codes, "params": params, "weights": w, "page_table": table, "kv_lens": lens, "budget": 8}
    for name, bad in (("weights", w[:5]), ("page_table", lens), ("new_table", lens), ("budget", 0), ("new_table", table[:1]),
                      ("new_lens", lens[:1]), ("weights", w.cpu()), ("codes", codes[0])):
        with pytest.raises(ValueError, match=name):
            capi.kv_cache_evict(**{**ok, name: bad})
    for name, bad in (("weights", w.double()), ("kept", w), ("new_lens", lens.long())):
        with pytest.raises(TypeError, match=name):
            capi.kv_cache_evict(**{**ok, name: bad})
    with pytest.raises(capi.I8qlError):
        capi.kv_cache_evict(**ok, first=5, last=4)
    with pytest.raises(capi.I8qlError):
        capi.kv_cache_evict(**ok, new_lens=lens)


# ------------------------------------------------------------------ eviction

def _scores(rng, shape, kind):
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 4, shape).astype(np.float32)
    elif kind == "signs":  # negative, both zeros, infinities, not a number
        w = rng.standard_normal(shape).astype(np.float32)
        pick = rng.integers(0, 8, shape)
        for i, v in enumerate((0.0, -0.0, np.inf, -np.inf, np.nan)):
            w[pick == i] = v
    elif kind == "near":  # equal but for the last bits
        w = (np.float32(1.0).view(np.uint32) + rng.integers(0, 3, shape).astype(np.uint32)).view(np.float32)
    elif kind == "same":
        w[:] = 0.25
    return w


def _evict(c, kind, budget, first, last, in_place, extra=0):
    """One eviction of a Cache (with room for the new pages), held to the oracle bit for bit."""
    rng = c.rng
    w = _scores(rng, (c.pages, c.heads, c.page), kind)
    weights = torch.from_numpy(w).cuda()
    args, _ = c.gpu()
    new = [min(n, budget) for n in c.lens]
    table, page = c.table, c.page
    if not in_place:
        need = [-(-n // page) for n in new]
        used = set(table[table >= 0].tolist())
        free = [p for p in range(c.pages) if p not in used]
        assert len(free) >= sum(need)
        table, at = np.full((len(new), max([*need, 1]) + extra), -9, np.int32), 0
        for i, n in enumerate(need):
            table[i, :n] = free[at:at + n]
            at += n
    codes, params = c.codes.cpu(), c.params.cpu().view(torch.int16)
    got_lens, kept = capi.kv_cache_evict(args["codes"], args["params"], weights, args["page_table"], args["kv_lens"], budget,
                                         first=first, last=last, new_table=None if in_place else torch.from_numpy(table).cuda())
    assert got_lens.tolist() == new
    want_codes, want_params, want_w = codes.clone(), params.clone(), w.copy()
    want_kept = np.full((len(new), c.heads, budget), -1, np.int32)
    for i, n in enumerate(c.lens):
        for h in range(c.heads):
            j = np.arange(n)
            mine = oracle.choose(w[c.table[i, j // page], h, j % page], n, budget, first, last)
            want_kept[i, h, : len(mine)] = mine
            s = np.arange(len(mine))
            to, src = (table[i, s // page], s % page), (c.table[i, mine // page], mine % page)
            want_codes[to[0], :, h, to[1]] = codes[src[0], :, h, src[1]]
            want_params[to[0], :, h, to[1]] = params[src[0], :, h, src[1]]
            want_w[to[0], h, to[1]] = w[src[0], h, src[1]]
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert torch.equal(c.codes.cpu(), want_codes) and torch.equal(c.params.cpu().view(torch.int16), want_params)
    assert np.array_equal(weights.cpu().numpy().view(np.uint32), want_w.view(np.uint32))
    return kept, table


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d,bits", [(64, 4), (128, 4), (64, 8), (128, 8)])
@pytest.mark.parametrize("lens,heads,page,budget,first,last,kind", [
    ([1], 1, 16, 1, 0, 0, "plain"),
    ([2], 2, 16, 1, 0, 1, "plain"),
    ([300, 0, 40, 41, 17], 3, 16, 40, 4, 16, "plain"),
    ([1000, 999, 64], 2, 64, 65, 0, 0, "ties"),
    ([500, 123], 5, 32, 100, 1, 99, "plain"),          # nothing to choose
    ([2500, 77], 2, 128, 1300, 4, 100, "signs"),
    ([3000], 1, 256, 2999, 0, 0, "near"),
    ([1025, 1024, 1023], 2, 16, 512, 3, 7, "same"),
])
def test_evict(lens, heads, page, budget, first, last, kind, d, bits, in_place):
    c = Cache(lens, heads, heads, d, bits, page, seed=budget + d, spare=2 + sum(-(-min(n, budget) // page) for n in lens))
    _evict(c, kind, budget, first, last, in_place, extra=d // 64)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,budget", [(20000, 5000), (70000, 300), (140001, 70000)])
def test_evict_long(n, budget, in_place):
    c = Cache([n, 60], 1, 1, 64, 4, 256, seed=n, spare=2 + budget // 256 + 3)
    _evict(c, "ties" if n == 20000 else "plain", budget, 4, 64, in_place)


def test_evict_many_sequences():
    c = Cache([17 + i for i in range(200)], 2, 2, 64, 4, 16, seed=1, spare=700)
    _evict(c, "plain", 33, 2, 9, False)


def test_evict_bad_input_is_recorded():
    def fresh():
        return Cache([300, 90], 2, 2, 64, 4, 16, seed=2, spare=20)
    c = fresh()
    args, _ = c.gpu()
    w = torch.rand((c.pages, 2, 16), device="cuda")
    before = (c.codes.clone(), c.params.clone(), w.clone())
    for entry, bad in ((1, -1), (1, c.pages), (0, 1 << 30)):
        table = torch.from_numpy(c.table).clone()
        table[0, entry] = bad
        lens, _ = capi.kv_cache_evict(c.codes, c.params, w, table.cuda(), args["kv_lens"], 40,
                                      new_table=torch.full((2, 3), -1, dtype=torch.int32, device="cuda"))
        assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX and lens.tolist() == [40, 40]
        for x, y in zip((c.codes, c.params.view(torch.int16), w), before):
            assert torch.equal(x, y.view(torch.int16) if y.dtype == torch.bfloat16 else y)
    # too few new pages, and a length past the table
    free = torch.arange(c.pages, dtype=torch.int32)[~torch.isin(torch.arange(c.pages, dtype=torch.int32), torch.from_numpy(c.table))]
    capi.kv_cache_evict(c.codes, c.params, w, args["page_table"], args["kv_lens"], 40, new_table=free[:4].view(2, 2).cuda())
    assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX
    c = fresh()
    args, _ = c.gpu()
    lens = torch.tensor([1 << 20, -3], dtype=torch.int32).cuda()
    capi.kv_cache_evict(c.codes, c.params, w, args["page_table"], lens, 40)
    assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX


def test_evict_nothing_to_do():
    codes, params = capi.kv_cache_alloc(2, 1, 16, 64)
    table, lens = torch.zeros((0, 3), dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    new, kept = capi.kv_cache_evict(codes, params, torch.zeros((2, 1, 16), device="cuda"), table, lens, 5)
    assert new.shape == (0,) and kept.shape == (0, 1, 5)


@pytest.mark.parametrize("nqs", [[1, 1], [40, 70]])
def test_other_stream_and_graph(nqs):
    c = Cache([700, 333], 4, 2, 128, 4, 32, nqs, seed=9)
    want = c.weigh()
    side = torch.cuda.Stream()
    got = torch.full_like(want, -5.0)
    args, at = c.gpu()
    q = c.q.cuda()
    torch.cuda.synchronize()
    capi.kv_cache_weights(q, weights=got, q_offsets=at, max_q=max(nqs), stream=side, **args)
    side.synchronize()
    cut = got.clone()
    torch.cuda.synchronize()
    new, kept = capi.kv_cache_evict(weights=cut, budget=100, first=4, last=30, stream=side.cuda_stream, **args)
    side.synchronize()
    assert torch.equal(got, want) and new.tolist() == [100, 100]
    # captured, with lengths that change between replays
    c = Cache([700, 333], 4, 2, 128, 4, 32, nqs, seed=9)
    args, at = c.gpu()
    w = torch.zeros((c.pages, 2, 32), device="cuda")
    spare = torch.full((2, 4), -1, dtype=torch.int32)
    free = [p for p in range(c.pages) if p not in set(c.table.reshape(-1).tolist())]
    assert len(free) == 2
    spare[0, 0], spare[1, 0] = free
    spare = spare.cuda()
    lens = args.pop("kv_lens")
    graph = torch.cuda.CUDAGraph()
    new, kept = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 2, 32), dtype=torch.int32, device="cuda")
    with torch.cuda.graph(graph):
        capi.kv_cache_weights(q, weights=w, q_offsets=at, max_q=max(nqs), kv_lens=lens, **args)
        capi.kv_cache_evict(weights=w, budget=32, first=2, last=10, kv_lens=lens, new_table=spare, new_lens=new, kept=kept, **args)
    for now in ([700, 333], [699, 100], [650, 20]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = (w.clone(), new.clone(), kept.clone())
        w.zero_()
        capi.kv_cache_weights(q, weights=w, q_offsets=at, max_q=max(nqs), kv_lens=lens, **args)
        ref = capi.kv_cache_evict(weights=w, budget=32, first=2, last=10, kv_lens=lens, new_table=spare, **args)
        assert torch.equal(got[1], ref[0]) and torch.equal(got[2], ref[1])
        assert got[1].tolist() == [min(n, 32) for n in now]
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


def test_past_32_bits():
    """Pages more than 2^32 bytes of codes into the cache give what the first pages give."""
    heads, d, bits, page, pages = 8, 128, 8, 256, 8300
    codes, params = capi.kv_cache_alloc(pages, heads, page, d, bits)
    assert codes.numel() > 1 << 32
    weights = torch.zeros((pages, heads, page), device="cuda")
    table = capi.rotary_table(capi.rotary_frequencies(d), 1000)
    torch.manual_seed(0)
    k, v = (torch.randn((700, heads, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    got = []
    for first in (0, pages - 6):
        own = torch.arange(first, first + 3, dtype=torch.int32, device="cuda")[None]
        slots = first * page + torch.arange(700, device="cuda")
        capi.kv_cache_store_rotary(None, k, v, table, slots, codes, params)
        lens = torch.tensor([700], dtype=torch.int32, device="cuda")
        sums = []
        for nq in (1, 2, 9, 40):
            q = torch.randn((nq, 32, d), generator=torch.Generator(device="cuda").manual_seed(nq), device="cuda").to(torch.bfloat16)
            capi.kv_cache_weights(q, codes, params, own, lens, weights, q_offsets=torch.tensor([0, nq], dtype=torch.int32).cuda(),
                                  max_q=nq)
            sums.append(weights[first:first + 3].clone())
        new, kept = capi.kv_cache_evict(codes, params, weights, own, lens, 300, first=4, last=50, new_table=own + 3)
        capi.kv_cache_evict(codes, params, weights, own, lens, 200, first=4, last=50)
        back = capi.kv_cache_load(codes, params, torch.cat([(first + 3) * page + torch.arange(300), first * page + torch.arange(200)]).cuda(), d)
        got.append((*sums, kept, *back))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("interleaved", [False, True])
def test_run_together(interleaved, bits):
    """A serving loop: prompts in chunks and single tokens, rotated, stored, attended over and weighed; contexts over
    the budget are cut.  Kept tokens, values and attention are followed on the host."""
    torch.manual_seed(1)
    d, heads, hq, page, budget, first, last = 64, 2, 6, 16, 48, 2, 12
    table = capi.rotary_table(capi.rotary_frequencies(d, 1e4, "linear", 2.0), 400)
    codes, params = capi.kv_cache_alloc(24, heads, page, d, bits)
    weights = torch.full((24, heads, page), float("nan"), device="cuda")  # (reused pages need no clearing)
    pages = torch.randperm(24).to(torch.int32).view(2, 12).cuda()
    lens, position = [0, 0], [0, 0]
    held = [[np.zeros((0, d)) for _ in range(heads)] for _ in range(2)]  # keys that the host expects, per head
    for step, counts in enumerate([(90, 50), (30, 7), (1, 1), (1, 1), (1, 1)]):
        t = sum(counts)
        qkv = torch.randn((t, hq + 2 * heads, d), device="cuda").to(torch.bfloat16)
        q, k, v = qkv.split([hq, heads, heads], dim=1)
        at, slots = [], []
        for i, n in enumerate(counts):
            at += range(position[i], position[i] + n)
            slots += [int(pages[i, j // page]) * page + j % page for j in range(lens[i], lens[i] + n)]
            position[i] += n
            lens[i] += n
        at, slots = torch.tensor(at).cuda(), torch.tensor(slots).cuda()
        q = capi.kv_cache_store_rotary(q, k, v, table, slots, codes, params, positions=at, interleaved=interleaved)
        kb, _ = capi.kv_cache_load(codes, params, slots, d)
        kv_lens = torch.tensor(lens, dtype=torch.int32).cuda()
        offsets = torch.tensor([0, counts[0], t], dtype=torch.int32).cuda()
        out = capi.kv_cache_attention(q, codes, params, pages, kv_lens, q_offsets=offsets, max_q=max(counts))
        capi.kv_cache_weights(q, codes, params, pages, kv_lens, weights, previous=weights, q_offsets=offsets, max_q=max(counts))
        # what the cache holds of each sequence, and attention over it
        a = 0
        for i, n in enumerate(counts):
            j = torch.arange(lens[i])
            pi = pages[i].cpu().long()[j // page]
            c = cache_oracle.unpack(codes.cpu().numpy()[pi, :, :, j % page], bits).transpose(1, 0, 2, 3)
            pr = params.float().cpu().numpy()[pi, :, :, j % page].transpose(1, 0, 2, 3)
            o, bound = kv_reference.attended(q[a:a + n].double().cpu(), c, pr[..., 0], pr[..., 1], n, 0, d ** -0.5,
                                             max(counts) * (hq // heads) > 32, 2 ** (bits - 1))
            assert ((out[a:a + n].double().cpu() - o).abs() <= bound).all()
            values = cache_oracle.values(c[0], pr[0, ..., 0], pr[0, ..., 1])
            for h in range(heads):
                held[i][h] = np.concatenate([held[i][h], kb[a:a + n, h].double().cpu().numpy()])
                # (kb is rounded to bf16)
                assert (np.abs(values[:, h] - held[i][h]) <= 2.0 ** -8 * np.abs(values[:, h]) + 1e-30).all()
            a += n
        before = [weights[pages[i].long()].transpose(0, 1).reshape(heads, -1)[:, : lens[i]].cpu().numpy() for i in range(2)]
        assert all(np.isfinite(w).all() and (w >= 0).all() for w in before)
        if step in (0, 1, 3):
            new, kept = capi.kv_cache_evict(codes, params, weights, pages, kv_lens, budget, first=first, last=last)
            for i in range(2):
                for h in range(heads):
                    mine = oracle.choose(before[i][h], lens[i], budget, first, last)
                    assert kept[i, h, : len(mine)].tolist() == mine.tolist()
                    held[i][h] = held[i][h][mine]
                lens[i] = min(lens[i], budget)
            assert new.tolist() == lens
