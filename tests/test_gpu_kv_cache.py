"""GPU parity of the quantized key/value cache (store, load, attention)
against the numpy oracle, through the binding.

Bars:
 * codes, scales and low values of kv_cache_store, and the values of
   kv_cache_load: bit-exact;
 * attention: every element within
     2^-8 |o|                     one bf16 rounding of the output
     + 2^-8 sum_j p_j |v_j - c_j| the rounding of each weight p_j s_j to bf16
                                  (c_j: the value of the centred code zero)
     + 2 delta sum_j p_j |v_j|    the logits' error delta: fp32 accumulation
                                  over the channels of the biased codes,
                                  D / 16 MMA steps and the scaling, 16 of
                                  2^-22 = 2^-18 of the summed magnitudes
     + 2^-14 sum_j p_j |v_j|      exp2 and the fp32 sums over tokens
   with few query rows (max_q * G <= 32); with more, where K and V become
   fp16 (2^-11) with scale and low value, and so do the centres c_j,
     2^-8 |o| + 2^-11 sum_j p_j (2 |v_j| + |c_j|)   P, V and the centres of V
     + 2 delta sum_j p_j |v_j| + 2^-14 sum_j p_j |v_j|
     delta = 2^-11 (max_j sum_d |q_d| (|k_jd| + |c_j|)) + 2^-18 of the same
   (times the softmax scale);
   and in both cases 2^-32 n max_j |v_j| over the n tokens a row sees: weights
   become fp16 after scaling, which rounds those under 2^-22 of the largest to
   multiples of 2^-32 of it (only visible where a dominant token's value is 0);
   where p, v and o are the 64-bit oracle's; and the whole output within
   4e-3 relative Frobenius (two bf16 roundings, 1.7e-3 rms each, with room).
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import capi
from oracle import kv_cache as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    from int8_quantized_linear_gb300 import build
    build.build()
    capi.lib()
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    yield
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


def _rows(rng, *shape):
    """bf16 values of widely varying rows: constants, exact ties, tiny and large magnitudes, outlier channels."""
    x = rng.standard_normal(shape).astype(np.float32)
    flat = x.reshape(-1, shape[-1])
    n = len(flat)
    flat[:, rng.integers(0, shape[-1])] *= 20
    for i, kind in enumerate(rng.integers(0, 12, n)):
        if kind == 0:
            flat[i] = rng.standard_normal()
        elif kind == 1:
            flat[i] *= np.float32(2.0 ** rng.integers(-125, 100))
        elif kind == 2:
            flat[i] = rng.integers(-8, 9, shape[-1]) / 2
        elif kind == 3:
            flat[i] = rng.integers(-30, 31, shape[-1])
            flat[i, :2] = [-30, 30]
        elif kind == 4:
            flat[i] = 0
    return torch.from_numpy(x).to(torch.bfloat16)


def _cache(pages, h, page, d, bits):
    """A cache whose every byte is known: codes 0xA5, params NaN."""
    codes, params = capi.kv_cache_alloc(pages, h, page, d, bits)
    codes.fill_(0xA5)
    params.fill_(float("nan"))
    return codes, params


def _host(codes, params, d):
    bits = codes.shape[-1] * 8 // d
    c = oracle.unpack(codes.cpu().numpy(), bits)
    p = params.float().cpu().numpy()
    return c, p[..., 0], p[..., 1]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t,h,page,fused", [(1, 1, 16, False), (1, 8, 64, True), (33, 3, 32, True), (257, 5, 256, False),
                                            (700, 16, 128, True)])
def test_store_and_load(bits, d, t, h, page, fused):
    rng = np.random.default_rng(t + d + bits)
    k, v = _rows(rng, t, h, d), _rows(rng, t, h, d)
    pages = -(-t // page) + 4
    slots = rng.permutation(pages * page)[:t].astype(np.int64)
    slots[rng.random(t) < 0.1] = -1 - rng.integers(0, 1 << 40)
    slots[0] = pages * page - 1 if (slots != pages * page - 1).all() else slots[0]
    codes, params = _cache(pages, h, page, d, bits)
    kd, vd = k.cuda(), v.cuda()
    if fused:  # slices of a wider row, as a fused projection leaves them
        wide = torch.full((t, 2 * h + 3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 3:3 + h], wide[:, 3 + h:] = kd, vd
        kd, vd = wide[:, 3:3 + h], wide[:, 3 + h:]
    sd = torch.from_numpy(slots).cuda()
    capi.kv_cache_store(kd, vd, sd, codes, params)
    kb, vb = capi.kv_cache_load(codes, params, sd, d)
    want_c = np.full((pages, 2, h, page, d * bits // 8), 0xA5, np.uint8)
    want_s = np.full((pages, 2, h, page, 2), np.nan, np.float32)
    back = np.zeros((2, t, h, d))
    live = slots >= 0
    for kv, x in enumerate((k, v)):
        c, s, low = oracle.quantize(x.float().numpy(), bits)
        at, off = slots[live] // page, slots[live] % page
        want_c[at, kv, :, off] = oracle.pack(c, bits)[live]
        want_s[at, kv, :, off] = np.stack([s, low], -1)[live]
        back[kv][live] = oracle.values(c, s, low)[live]
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(params.float().cpu().numpy(), want_s, equal_nan=True)
    for kv, got in enumerate((kb, vb)):
        # low + s * c in fp32 (s * c is exact), then bf16: two roundings, both reproduced
        want = torch.from_numpy(back[kv].astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("bits,d", [(4, 128), (8, 64)])
@pytest.mark.parametrize("ahead", [8, 16, 24])
def test_load_into_any_16_byte_boundary(bits, d, ahead):
    t, h, page = 77, 3, 16
    rng = np.random.default_rng(ahead)
    codes, params = _cache(6, h, page, d, bits)
    x = _rows(rng, t, h, d).cuda()
    slots = torch.from_numpy(rng.permutation(6 * page)[:t].astype(np.int64)).cuda()
    capi.kv_cache_store(x, -x, slots, codes, params)
    want = capi.kv_cache_load(codes, params, slots, d)
    room = torch.full((2, t * h * d + 48), 7.0, dtype=torch.bfloat16, device="cuda")
    kb, vb = (r[n:n + t * h * d].view(t, h, d) for r, n in zip(room, (ahead, 16)))
    capi.kv_cache_load(codes, params, slots, d, k=kb, v=vb)
    assert torch.equal(kb, want[0]) and torch.equal(vb, want[1])
    for r, n in zip(room, (ahead, 16)):
        assert (r[:n] == 7).all() and (r[n + t * h * d:] == 7).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_codes_are_the_rounded_quotients(bits):
    """A million rows' worth of quotients over all scales a row can have, ties and their neighbours among them."""
    t, h, d, page = 1024, 8, 128, 64
    rng = np.random.default_rng(bits)
    x = rng.integers(-255, 256, (t, h, d)).astype(np.float32) * np.exp2(rng.integers(-8, 9, (t, h, 1)).astype(np.float32))
    x *= np.exp2(rng.integers(-120, 110, (t, h, 1)).astype(np.float32))
    x[::2] += np.abs(x[::2]).max(-1, keepdims=True) * rng.uniform(-4, 4, (t // 2, h, 1)).astype(np.float32)
    k = torch.from_numpy(x).to(torch.bfloat16)
    v = torch.from_numpy(rng.permutation(x.ravel()).reshape(x.shape)[..., :]).to(torch.bfloat16)
    codes, params = _cache(t // page, h, page, d, bits)
    capi.kv_cache_store(k.cuda(), v.cuda(), torch.arange(t, device="cuda"), codes, params)
    got_c, got_s, got_low = _host(codes, params, d)
    for kv, y in enumerate((k, v)):
        c, s, low = oracle.quantize(y.float().numpy(), bits)
        shape = lambda a: np.moveaxis(a.reshape(t // page, page, h, *a.shape[2:]), 1, 2)  # noqa: E731
        assert np.array_equal(got_c[:, kv], shape(c))
        assert np.array_equal(got_s[:, kv], shape(s)) and np.array_equal(got_low[:, kv], shape(low))


def test_store_takes_non_finite_rows_without_touching_others():
    t, h, d, page = 6, 2, 128, 16
    rng = np.random.default_rng(0)
    k = torch.from_numpy(rng.standard_normal((t, h, d))).to(torch.bfloat16)
    bad = k.clone()
    bad[1, 0, 5], bad[2, 1, 0], bad[4, 0] = float("nan"), float("inf"), float("-inf")
    slots = torch.arange(t, device="cuda")
    a, b = _cache(1, h, page, d, 4), _cache(1, h, page, d, 4)
    capi.kv_cache_store(k.cuda(), k.cuda(), slots, *a)
    capi.kv_cache_store(bad.cuda(), k.cuda(), slots, *b)
    same = torch.ones(2, h, page, dtype=torch.bool)
    for i, j in ((1, 0), (2, 1), (4, 0)):
        same[0, j, i] = False
    assert torch.equal(a[0].cpu()[0][same], b[0].cpu()[0][same])
    assert torch.equal(a[1].cpu()[0][same].view(torch.int16), b[1].cpu()[0][same].view(torch.int16))


def test_slots_past_the_cache_are_reported():
    codes, params = _cache(2, 1, 16, 64, 4)
    k = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 32, 1 << 50], device="cuda")
    capi.kv_cache_store(k, k, slots, codes, params)
    assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX
    assert (codes[1] == 0xA5).all()
    kb, _ = capi.kv_cache_load(codes, params, slots, 64)
    assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX
    assert (kb[0] == 1).all() and not kb[1:].any()
    capi.kv_cache_store(k[:0], k[:0], slots[:0], codes, params)  # nothing to do


# ------------------------------------------------------------------ attention

class Problem:
    """A paged cache of random codes around sequences of the given lengths,
    with NaN wherever nothing was written."""

    def __init__(self, lens, nqs, hq, h, d, bits, page, seed, spare=3, spread=1.0, offset=0.0):
        rng = np.random.default_rng(seed)
        self.lens, self.nqs, self.d, self.bits, self.page = lens, nqs, d, bits, page
        need = [-(-n // page) for n in lens]
        pages, wide = sum(need) + spare, max(need + [1]) + 1
        order = rng.permutation(pages)
        table = np.full((len(lens), wide), -1, np.int32)
        levels = 2 ** bits - 1
        c = rng.integers(0, levels + 1, (pages, 2, h, page, d)).astype(np.uint8)
        s = (2.0 * spread / levels * rng.uniform(0.7, 1.4, (pages, 2, h, page))).astype(np.float32)
        low = (-s * levels / 2 * rng.uniform(0.8, 1.2, s.shape) + offset).astype(np.float32)
        params = torch.from_numpy(np.stack([s, low], -1)).to(torch.bfloat16)
        self.seqs, at = [], 0
        written = np.zeros((pages, page), bool)
        for b, n in enumerate(lens):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            if n:
                written[table[b, :need[b]]] = True
                written[table[b, need[b] - 1], (n - 1) % page + 1:] = False
        p = params.float().numpy()
        for b, n in enumerate(lens):
            pg = table[b, :need[b]]
            pick = lambda x: np.moveaxis(x[pg], 0, 2).reshape(2, h, need[b] * page, *x.shape[4:])[:, :, :n].swapaxes(1, 2)  # noqa: E731
            self.seqs.append((pick(c), pick(p[..., 0]), pick(p[..., 1])))
        params[torch.from_numpy(~written)[:, None, None].expand(pages, 2, h, page)] = float("nan")
        self.codes = torch.from_numpy(oracle.pack(c, bits)).cuda()
        self.params = params.cuda()
        self.q = torch.from_numpy(rng.standard_normal((sum(nqs), hq, d)) * spread).to(torch.bfloat16)
        self.table, self.kv_lens = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(nqs)]), dtype=torch.int32).cuda()

    def run(self, window=0, scale=None, q=None, single=None, max_q="known", **kw):
        single = all(n == 1 for n in self.nqs) if single is None else single
        hint = 1 if single else max(self.nqs + [1]) if max_q == "known" else max_q or self.q.shape[0]
        self.wide = hint * self.q.shape[1] // self.codes.shape[2] > 32
        if not single:
            kw["q_offsets"] = self.offsets
            kw["max_q"] = max(self.nqs + [1]) if max_q == "known" else max_q
        return capi.kv_cache_attention(self.q.cuda() if q is None else q, self.codes, self.params, self.table,
                                       self.kv_lens, window=window, scale=scale, **kw)

    def check(self, y, window=0, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        y, q, at = y.double().cpu().numpy(), self.q.double().numpy(), 0
        assert np.isfinite(y).all()
        err = ref = 0.0
        for (c, s, low), nq in zip(self.seqs, self.nqs):
            a = oracle.attention(q[at:at + nq], c, s, low, nq, window, scale, centre=2 ** (self.bits - 1))
            got = y[at:at + nq]
            at += nq
            if self.wide:
                bound = 2.0 ** -8 * np.abs(a.out) + 2.0 ** -11 * (2 * a.size + a.mid) + a.size * (
                    2.0 ** -10 * (a.logit + a.mid_logit)[..., None] * (1 + 2.0 ** -7) + 2.0 ** -14) + 1e-37
            else:
                bound = 2.0 ** -8 * (np.abs(a.out) + a.weighted) + a.size * (
                    2.0 ** -17 * a.biased[..., None] + 2.0 ** -14) + 1e-37
            bound = bound + 2.0 ** -32 * a.flush
            off = np.abs(got - a.out)
            assert np.all(off <= bound), f"off by {np.max(off / bound):.3g} of the bound"
            err += np.sum(off ** 2)
            ref += np.sum(a.out ** 2)
        if y.size >= 1024:
            assert err <= (4e-3) ** 2 * ref, f"relative error {np.sqrt(err / ref):.2e}"


LAYOUTS = [(32, 8, 128), (4, 4, 128), (7, 1, 64), (10, 2, 128), (24, 3, 64), (16, 1, 128), (20, 1, 64)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hq,h,d", LAYOUTS)
def test_single_tokens(hq, h, d, bits):
    """One query token per sequence, lengths from none and one to several tiles."""
    p = Problem([1, 0, 2, 15, 16, 17, 127, 128, 129, 300, 1025, 31], [1] * 12, hq, h, d, bits, 16, hq + d + bits)
    p.check(p.run())


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("bits", [4, 8])
def test_page_sizes(page, bits):
    p = Problem([page - 1, page, page + 1, 5 * page + 3, 700], [1] * 5, 8, 2, 128, bits, page, page)
    p.check(p.run())


@pytest.mark.parametrize("window", [1, 17, 128, 129, 1000])
@pytest.mark.parametrize("bits", [4, 8])
def test_windows(window, bits):
    p = Problem([1, 16, 130, 555, 2000], [1] * 5, 8, 2, 64, bits, 32, window)
    p.check(p.run(window=window), window=window)


def test_pages_before_the_window_are_not_read():
    p = Problem([1500, 900], [1, 1], 8, 2, 128, 4, 16, 5)
    y = p.run(window=100)
    p.check(y, window=100)
    p.table[0, :(1500 - 100) // 16] = -1
    p.table[1, :(900 - 100) // 16] = 1 << 30
    assert torch.equal(p.run(window=100), y)
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hq,h,d", [(8, 2, 128), (7, 1, 64), (3, 3, 128), (16, 1, 64)])
@pytest.mark.parametrize("window", [0, 40])
def test_drafts(hq, h, d, bits, window):
    """A few query tokens per sequence, none for some, more than the cache has for others."""
    nqs = [1, 0, 5, 3, 0, 8, 4, 2, 6]
    p = Problem([9, 40, 5, 129, 0, 300, 2, 0, 131], nqs, hq, h, d, bits, 16, hq + bits)
    y = p.run(window=window)
    p.check(y, window=window)
    assert not y[9:9 + 5][0:0].any()
    # rows that see nothing are exactly zero: the first queries of the sequences with 2 and 0 tokens
    start = np.concatenate([[0], np.cumsum(nqs)])
    assert not y[start[6]:start[6] + 2].any() and not y[start[7]:start[8]].any()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hq,h,d", [(8, 2, 128), (8, 2, 64), (3, 3, 128), (7, 1, 64), (20, 1, 128)])
@pytest.mark.parametrize("window", [0, 150])
def test_prompts(hq, h, d, bits, window):
    """Prompt chunks: lengths around tiles and row blocks, whole prompts and chunks behind a cached prefix, beside
    single tokens and empty sequences."""
    nqs = [130, 64, 1, 0, 33, 129, 7]
    p = Problem([130, 300, 411, 50, 33, 700, 5], nqs, hq, h, d, bits, 16, hq + bits + window)
    y = p.run(window=window)
    p.check(y, window=window)
    assert torch.equal(p.run(window=window), y)
    start = np.concatenate([[0], np.cumsum(nqs)])
    assert not y[start[6]:start[6] + 2].any()  # five tokens, seven queries: the first two see nothing


@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("bits", [4, 8])
def test_prompt_over_a_long_prefix(page, bits):
    """Few row blocks over many tiles: cut between CTAs and joined."""
    p = Problem([5003, 900], [40, 70], 8, 2, 128, bits, page, page + bits)
    y = p.run()
    p.check(y)
    assert torch.equal(p.run(), y)


@pytest.mark.parametrize("spread,offset", [(8.0, 0.0), (1e-6, 0.0), (1.0, 30.0), (1e4, 0.0)])
def test_prompt_value_ranges(spread, offset):
    p = Problem([400, 300], [90, 70], 8, 2, 128, 4, 16, 14, spread=spread, offset=offset)
    scale = p.d ** -0.5 / (spread if spread > 100 else 1)
    p.check(p.run(scale=scale), scale=scale)


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_prompt_negative_and_zero_scale(scale):
    p = Problem([300], [80], 4, 2, 64, 8, 16, 18)
    p.check(p.run(scale=scale), scale=scale)


@pytest.mark.parametrize("nq", [1, 60])
def test_values_of_growing_size(nq):
    """Scales that grow by far along the context: the sums are brought to the larger unit."""
    p = Problem([1100], [nq], 8, 2, 128, 4, 16, 21)
    c, s, low = p.seqs[0]
    grow = np.exp2(np.arange(1100) // 64 * 3.0 - 30).astype(np.float32)[None, :, None]
    grow = np.concatenate([np.ones_like(grow), grow])
    p.seqs[0] = (c, s * grow, low * grow)
    pages = p.table[0, :-(-1100 // 16)].long()
    full = torch.ones(len(pages) * 16)
    full[:1100] = torch.from_numpy(grow[1, :, 0])
    p.params[pages, 1] = (p.params[pages, 1].float() * full.view(-1, 1, 16, 1).cuda()).to(torch.bfloat16)
    p.check(p.run())


@pytest.mark.parametrize("nq", [1, 60])
def test_non_finite_queries_stay_in_their_rows(nq):
    p = Problem([200], [nq], 8, 2, 128, 4, 16, 22)
    want = p.run()
    q = p.q.clone()
    q[0, 1, 7], q[-1, 5, 3] = float("nan"), float("inf")
    y = p.run(q=q.cuda())
    assert torch.isnan(y[0, 1]).all() and torch.isnan(y[-1, 5]).any()
    keep = torch.ones(nq, 8, dtype=torch.bool)
    keep[0, 1] = keep[-1, 5] = False
    assert torch.equal(y.cpu()[keep], want.cpu()[keep])


def test_max_q_only_chooses_the_kernel():
    p = Problem([50, 400, 130], [2, 7, 1], 8, 4, 128, 4, 32, 9)
    for hint in (1, 2, 7, 1000, None):
        p.check(p.run(max_q=hint))


def test_single_token_form_equals_offsets():
    p = Problem([50, 400, 1300], [1, 1, 1], 8, 4, 128, 4, 32, 10)
    assert torch.equal(p.run(single=True), p.run(single=False))


@pytest.mark.parametrize("batch,most", [(159, 300), (161, 300), (400, 300), (641, 200), (1500, 150)])
def test_many_sequences(batch, most):
    rng = np.random.default_rng(batch)
    nqs = rng.integers(0, 3, batch).tolist()
    p = Problem(rng.integers(0, most, batch).tolist(), nqs, 4, 2, 64, 4, 16, batch)
    p.check(p.run())


def test_many_prompts():
    """More prompts than one round of the work sharing looks at, most of them empty."""
    rng = np.random.default_rng(0)
    nqs = [int(n) if rng.random() < 0.03 else 0 for n in rng.integers(1, 90, 2100)]
    p = Problem([n + int(rng.integers(0, 60)) for n in nqs], nqs, 4, 2, 64, 4, 16, 2100)
    p.check(p.run())


@pytest.mark.parametrize("lens", [[20011], [30000, 3], [5, 9000, 9001, 1]])
@pytest.mark.parametrize("bits", [4, 8])
def test_long_contexts_are_joined(lens, bits):
    p = Problem(lens, [1] * len(lens), 8, 2, 128, bits, 64, sum(lens))
    y = p.run()
    p.check(y)
    for _ in range(3):  # the order of the parts is fixed: the same bits every time
        assert torch.equal(p.run(), y)


@pytest.mark.parametrize("spread,offset", [(8.0, 0.0), (1e-6, 0.0), (1.0, 30.0), (1e4, 0.0)])
def test_value_ranges(spread, offset):
    """Peaked and flat softmaxes, tiny values, and values far from zero."""
    p = Problem([700, 64, 1, 258], [1, 2, 1, 3], 8, 2, 128, 4, 16, 4, spread=spread, offset=offset)
    scale = p.d ** -0.5 / (spread if spread > 100 else 1)
    p.check(p.run(scale=scale), scale=scale)


def test_negative_and_zero_scale():
    p = Problem([300, 20], [1, 1], 4, 2, 64, 8, 16, 8)
    for scale in (0.0, -0.2):
        p.check(p.run(scale=scale), scale=scale)


def test_strided_queries_streams_and_workspace():
    p = Problem([300, 2000, 47], [1, 4, 2], 8, 2, 128, 4, 16, 77)
    want = p.run()
    wide = torch.full((7, 12, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = p.q.cuda()
    assert torch.equal(p.run(q=wide[:, 2:10]), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    q = p.q.cuda()
    torch.cuda.synchronize()
    p.run(q=q, stream=st, out=out)
    st.synchronize()
    assert torch.equal(out, want)
    p.run(q=q, stream=st.cuda_stream, out=out.zero_())
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_workspace():
    """Contexts long enough to be cut between CTAs: a given workspace, with anything in it, and one too small."""
    p = Problem([300, 20000, 47], [1, 4, 2], 8, 2, 128, 4, 16, 77)
    want = p.run()
    size = capi.i8ql_kv_attention_workspace(3, 7, 8, 2, 128, 4, 16, p.table.shape[1], 4)
    assert size > 0
    ws = torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda")  # contents do not matter
    assert torch.equal(p.run(workspace=ws), want)
    with pytest.raises(capi.I8qlError) as err:
        p.run(workspace=ws[:size - 1])
    assert err.value.status == capi.I8QL_ERR_WORKSPACE_LIMIT


@pytest.mark.parametrize("width", [0, 80, 2000])
def test_page_table_width_only_chooses_the_form(width):
    """The same sequences behind a wider table: joined in clusters, by a second kernel, or not cut at all."""
    p = Problem([700, 1, 0, 300, 17], [1, 2, 1, 0, 1], 8, 2, 128, 4, 16, 31)
    p.table = torch.cat([p.table, torch.full((5, width), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    p.check(p.run())


def test_keys_with_outlier_channels():
    """Keys as models have them (a few channels many times the rest), stored and attended over: the whole output
    within 2.5e-3 of the fp64 attention over the quantized values (its own bf16 rounding is 1.7e-3 rms)."""
    n, h, d, page = 600, 2, 128, 64
    for bits in (4, 8):
        g = torch.Generator().manual_seed(bits)
        k = torch.randn((n, h, d), generator=g)
        k[..., [5, 77]] *= 60.0
        k, v = k.to(torch.bfloat16), torch.randn((n, h, d), generator=g).to(torch.bfloat16)
        codes, params = _cache(10, h, page, d, bits)
        capi.kv_cache_store(k.cuda(), v.cuda(), torch.arange(n, device="cuda"), codes, params)
        c, s, low = (np.stack(t) for t in zip(*(oracle.quantize(x.float().numpy(), bits) for x in (k, v))))
        for nq in (1, 3, 50):
            q = torch.randn((nq, 8, d), generator=g).to(torch.bfloat16)
            y = capi.kv_cache_attention(q.cuda(), codes, params, torch.arange(10, dtype=torch.int32, device="cuda")[None],
                                        torch.tensor([n], dtype=torch.int32, device="cuda"),
                                        q_offsets=torch.tensor([0, nq], dtype=torch.int32, device="cuda"), max_q=nq)
            ref = oracle.attention(q.double().numpy(), c, s, low, nq, 0, d ** -0.5).out
            assert np.linalg.norm(y.double().cpu().numpy() - ref) <= 2.5e-3 * np.linalg.norm(ref), (bits, nq)


def test_graph_capture():
    p = Problem([300, 2000, 47], [1, 1, 1], 8, 2, 128, 4, 16, 78)
    q, want = p.q.cuda(), p.run()
    out, graph = torch.zeros_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(q=q, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # lengths are read on the device: the same graph serves other lengths
    p.kv_lens.copy_(torch.tensor([299, 3, 20], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, p.run(q=q))


def test_sizes_out_of_range_are_reported():
    """Bad pages, lengths and offsets come back as a status, and rows of other sequences are right."""
    p = Problem([300, 200, 47], [2, 2, 2], 8, 2, 128, 4, 16, 79)
    want = p.run()
    for change in ("page", "negative page", "length", "negative length", "offset"):
        keep = [t.clone() for t in (p.table, p.kv_lens, p.offsets)]
        if change.endswith("page"):
            p.table[1, 3] = -5 if change.startswith("neg") else p.codes.shape[0]
        elif change.endswith("length"):
            p.kv_lens[1] = -7 if change.startswith("neg") else 1 << 30
            if change == "length":
                p.table[1] = p.table[1].clamp(min=0)
        else:
            p.offsets[1], p.offsets[2] = 1 << 20, -3
        y = p.run()
        assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX, change
        if change != "offset":
            assert torch.equal(y[:2], want[:2]) and torch.equal(y[4:], want[4:]), change
        p.table, p.kv_lens, p.offsets = keep
    assert torch.equal(p.run(), want)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes, written, read and attended over at its end."""
    page, h, d, n = 256, 16, 128, 300
    pages = (1 << 32) // (2 * h * page * d) + 40
    codes = torch.empty((pages, 2, h, page, d), dtype=torch.uint8, device="cuda")
    params = torch.empty((pages, 2, h, page, 2), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(5)
    k, v = ((torch.randn((n, h, d), generator=g)).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 30]], dtype=torch.int32)
    j = torch.arange(n)
    slots = (table[0, j // page].long() * page + j % page).cuda()
    capi.kv_cache_store(k.cuda(), v.cuda(), slots, codes, params)
    kb, vb = capi.kv_cache_load(codes, params, slots, d)
    c, s, low = zip(*(oracle.quantize(x.float().numpy(), 8) for x in (k, v)))
    for got, i in ((kb, 0), (vb, 1)):
        want = torch.from_numpy(oracle.values(c[i], s[i], low[i]).astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)
    q = torch.randn((1, h, d), generator=g).to(torch.bfloat16)
    y = capi.kv_cache_attention(q.cuda(), codes, params, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    ref = oracle.attention(q.double().numpy(), np.stack(c), np.stack(s), np.stack(low), 1, 0, d ** -0.5, centre=128)
    bound = 2.0 ** -8 * (np.abs(ref.out) + ref.weighted) + ref.size * (2.0 ** -17 * ref.biased[..., None] + 2.0 ** -14)
    assert np.all(np.abs(y.double().cpu().numpy() - ref.out) <= bound)
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
