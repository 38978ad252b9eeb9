"""GPU tests of rotary positions through the binding: tables against the angle
of the exact product, rows and the rotated store bit for bit against the
contract's fp32 operations, gradients, strides, padding, streams and graphs."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import capi
from oracle import rotary as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    from int8_quantized_linear_gb300 import build
    build.build()
    capi.lib()
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    yield
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


def _bits(t):
    return t.contiguous().view(torch.int16).cpu()


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def _table(rows, rot, seed=0):
    """Any numbers do for what turns rows: not only cosines and sines."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, rot), generator=g)


def _rows(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16)


# The angle's fraction of a turn keeps 2^-29 turns at least (24 bits of an eighth), and
# what the fixed point leaves for |p| < 2^31; the function's own error is within 2 ulp, and
# the amplitude rounds once: 2^-29 2 pi + 2 * 2^-24 + 2^-24 < 2^-22 of the amplitude.
@pytest.mark.parametrize("n,f", [(1, 1), (7, 3), (40, 64), (33, 24), (300, 256), (65, 128)])
def test_table(n, f):
    rng = np.random.default_rng(n)
    freqs = np.exp(-rng.random(f) * 14)
    freqs[0] = 1.0
    at = rng.integers(0, 1 << 20, n)
    at[: 6] = np.array([0, 1, -1, (1 << 31) - 1, -(1 << 30), 12345])[: len(at[:6])]
    for amplitude in (1.0, 1.375):
        got = capi.rotary_table(torch.from_numpy(freqs).cuda(), torch.from_numpy(at).cuda(), amplitude).cpu().double()
        ref = torch.from_numpy(oracle.table(freqs, at, amplitude))
        assert got.shape == (n, 2 * f)
        assert float((got - ref).abs().max()) <= 2.0 ** -22 * amplitude
    # near 0 the sine keeps its relative precision
    small = torch.tensor([1e-9, 3e-7], dtype=torch.float64)
    s = capi.rotary_table(small.cuda(), 4).cpu().double()[:, 2:]
    want = torch.sin(torch.arange(4, dtype=torch.float64)[:, None] * small)
    assert ((s - want).abs() <= 2.0 ** -21 * want).all()


# Frequencies of either sign, to the same bound (see test_table), whatever their size.
def test_table_signs():
    freqs = np.array([-1e-4, -3e-13, -0.7, -6.3, -1e5, 2e5, 1e-13, -1.0])
    at = np.array([0, 1, -1, (1 << 31) - 1, -(1 << 31) + 1, 77777])
    got = capi.rotary_table(torch.from_numpy(freqs).cuda(), torch.from_numpy(at).cuda()).cpu().double()
    assert float((got - torch.from_numpy(oracle.table(freqs, at))).abs().max()) <= 2.0 ** -22
    # near 0 the sine keeps its relative precision: 2^-55 turns that are cut off, of 2^-32.6 and
    # more, and the series' and products' roundings, 2^-22.4 + 2^-24 + 2^-24
    small = torch.tensor([-1e-9, -3e-7], dtype=torch.float64)
    s = capi.rotary_table(small.cuda(), 4).cpu().double()[:, 2:]
    want = torch.sin(torch.arange(4, dtype=torch.float64)[:, None] * small)
    assert ((s - want).abs() <= 2.0 ** -21 * want.abs()).all()


@pytest.mark.parametrize("n", [0, 1, 5, 1000, 70001])
def test_table_range(n):
    f = capi.rotary_frequencies(96, 10000.0)
    table = torch.full((n + 1, 96), 7.0, device="cuda")
    out = capi.rotary_table(f, n, table=table[:n])
    assert n == 0 or out.data_ptr() == table.data_ptr()
    ref = torch.outer(torch.arange(n, dtype=torch.float64), f.cpu())
    ref = torch.cat([torch.cos(ref), torch.sin(ref)], 1)
    assert n == 0 or float((out.cpu().double() - ref).abs().max()) <= 2.0 ** -22
    assert (table[n] == 7.0).all()


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,heads,d,rot", [(1, 1, 8, 8), (1, 40, 128, 128), (5, 3, 72, 24), (33, 5, 80, 32), (7, 2, 512, 512),
                                           (70, 16, 96, 48), (130, 7, 64, 16), (6, 1, 72, 72), (2100, 9, 128, 64)])
def test_apply(t, heads, d, rot, interleaved, backward):
    x, table = _rows(t, t, heads, d), _table(50, rot)
    g = torch.Generator().manual_seed(t)
    at = torch.randint(0, 50, (t,), generator=g)
    want = _bf16(oracle.turn(x.float().numpy(), table[at].numpy(), interleaved, backward))
    got = capi.rotary_apply(x.cuda(), table.cuda(), at.cuda(), interleaved=interleaved, backward=backward)
    assert torch.equal(_bits(got), _bits(want))
    # a slice of wider rows, into a slice of wider rows, whose other columns stay
    wide = torch.full((t, heads + 3, d), 5.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((t, heads + 2, d), 6.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:1 + heads] = x.cuda()
    back = capi.rotary_apply(wide[:, 1:1 + heads], table.cuda(), at.cuda(), interleaved=interleaved, backward=backward,
                             out=out[:, :heads])
    assert back.data_ptr() == out.data_ptr()
    assert torch.equal(_bits(out[:, :heads]), _bits(want)) and (out[:, heads:] == 6.0).all()
    # in place
    capi.rotary_apply(wide[:, 1:1 + heads], table.cuda(), at.cuda(), interleaved=interleaved, backward=backward,
                      out=wide[:, 1:1 + heads])
    assert torch.equal(_bits(wide[:, 1:1 + heads]), _bits(want))
    assert (wide[:, 0] == 5.0).all() and (wide[:, 1 + heads:] == 5.0).all()


def test_apply_rows_in_order_and_padding():
    x, table = _rows(3, 40, 4, 64).cuda(), _table(60, 64).cuda()
    assert torch.equal(_bits(capi.rotary_apply(x, table)), _bits(capi.rotary_apply(x, table, torch.arange(40).cuda())))
    at = torch.arange(40)
    at[::3] = -1 - torch.arange(14) * (1 << 40)
    y = capi.rotary_apply(x, table, at.cuda())
    assert torch.equal(_bits(y[::3]), _bits(x[::3]))
    assert torch.equal(_bits(y[at >= 0]), _bits(capi.rotary_apply(x, table)[at >= 0]))
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    for bad in (60, 1 << 40, (1 << 63) - 1):
        at[5] = bad
        y = capi.rotary_apply(x, table, at.cuda())
        assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX
        assert torch.equal(_bits(y[5]), _bits(x[5]))
    assert capi.rotary_apply(x[:0], table).shape == (0, 4, 64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_is_the_gradient(interleaved):
    t, heads, d, rot = 37, 3, 48, 32
    f = capi.rotary_frequencies(rot, 500.0)
    table = capi.rotary_table(f, torch.arange(1000, 1000 + t).cuda(), 1.25)
    x, g = _rows(1, t, heads, d), _rows(2, t, heads, d)
    got = capi.rotary_apply(g.cuda(), table, interleaved=interleaved, backward=True).cpu().double()
    rows = table.cpu().double().numpy()
    # the formula's, rounded to bf16 once after fp32 (three roundings of 2^-24 on magnitudes up to 1.25 (|a| + |b|))
    want = torch.from_numpy(oracle.turn64(g.double().numpy(), rows, interleaved, True))
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * 1.25 * 2 * float(g.float().abs().max())).all()
    # and by differences: the function is linear, so any step is exact but for 64-bit rounding
    rng = np.random.default_rng(0)
    for _ in range(20):
        i, h, c = rng.integers(0, t), rng.integers(0, heads), rng.integers(0, d)
        step = np.zeros((t, heads, d))
        step[i, h, c] = 0.5
        lo, hi = (oracle.turn64(x.double().numpy() + s * step, rows, interleaved) for s in (-1, 1))
        slope = float(((hi - lo) * g.double().numpy()).sum())
        assert math.isclose(slope, float(want[i, h, c]), rel_tol=1e-9, abs_tol=1e-9)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,hq,h,d,rot,page,fused", [(1, 4, 1, 64, 64, 16, False), (1, 32, 8, 128, 128, 64, True),
                                                     (45, 0, 3, 64, 16, 32, False), (33, 7, 1, 128, 64, 256, True),
                                                     (700, 6, 6, 64, 32, 16, True), (300, 15, 5, 128, 128, 128, False)])
def test_store_rotary(t, hq, h, d, rot, page, fused, interleaved, bits):
    """Bit for bit what rotating and then storing gives, whose parts are tested by themselves."""
    qkv = _rows(t + d, t, hq + 2 * h, d).cuda()
    qkv[:, :, 3] *= 30
    q, k, v = qkv.split([hq, h, h], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    table = _table(90, rot).cuda()
    g = torch.Generator().manual_seed(t)
    at = torch.randint(0, 90, (t,), generator=g)
    at[torch.rand(t, generator=g) < 0.1] = -1
    pages = -(-t // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:t]
    slots[torch.rand(t, generator=g) < 0.2] = -1
    at, slots = at.cuda(), slots.cuda()
    caches = []
    for _ in range(2):
        codes, params = capi.kv_cache_alloc(pages, h, page, d, bits)
        codes.fill_(0xA5)
        params.fill_(-3.0)
        caches.append((codes, params))
    out = capi.kv_cache_store_rotary(q if hq else None, k, v, table, slots, *caches[0], positions=at, interleaved=interleaved)
    turned = capi.rotary_apply(k, table, at, interleaved=interleaved)
    capi.kv_cache_store(turned, v, slots, *caches[1])
    for a, b in zip(*caches):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    if hq == 0:
        assert out is None
        return
    want = capi.rotary_apply(q, table, at, interleaved=interleaved)
    assert torch.equal(_bits(out), _bits(want))
    # the queries in place
    kept = qkv[:, hq:].clone()
    back = capi.kv_cache_store_rotary(q, k, v, table, slots, *caches[0], positions=at, interleaved=interleaved, q_out=q)
    assert back.data_ptr() == q.data_ptr() and torch.equal(_bits(q), _bits(want))
    assert torch.equal(_bits(qkv[:, hq:]), _bits(kept))


def test_store_rotary_past_the_end():
    k = _rows(9, 4, 2, 64).cuda()
    codes, params = capi.kv_cache_alloc(2, 2, 16, 64)
    codes.fill_(0xA5)
    before = codes.clone()
    table = _table(8, 64).cuda()
    capi.kv_cache_store_rotary(None, k, k, table, torch.tensor([32, 1 << 50, 33, -1]).cuda(), codes, params)
    assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX
    assert torch.equal(codes, before)
    # a position past the table: stored as it is
    capi.kv_cache_store_rotary(None, k, k, table, torch.arange(4).cuda(), codes, params,
                               positions=torch.tensor([8, 9, 10, 1 << 40]).cuda())
    assert capi.i8ql_get_device_error() == capi.I8QL_ERR_BAD_INDEX
    other, op = torch.empty_like(codes), torch.empty_like(params)
    capi.kv_cache_store(k, k, torch.arange(4).cuda(), other, op)
    assert torch.equal(codes[0, :, :, :4], other[0, :, :, :4])


def test_other_stream_and_graph():
    x, table, at = _rows(4, 600, 8, 128).cuda(), _table(600, 128).cuda(), torch.arange(599, -1, -1).cuda()
    want = capi.rotary_apply(x, table, at)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = capi.rotary_apply(x, table, at, stream=side)
    side.synchronize()
    assert torch.equal(_bits(got), _bits(want))
    f = capi.rotary_frequencies(128)
    pos, buf, out = torch.zeros(600, dtype=torch.int64, device="cuda"), torch.empty((600, 128), device="cuda"), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.rotary_table(f, pos, table=buf)
        capi.rotary_apply(x, buf, out=out)
    for begin in (5, 100000):
        pos.copy_(torch.arange(begin, begin + 600))
        graph.replay()
        torch.cuda.synchronize()
        ref = capi.rotary_apply(x, capi.rotary_table(f, pos))
        assert torch.equal(_bits(out), _bits(ref))


def test_binding_refusals():
    x, table = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((10, 64), device="cuda")
    at = torch.zeros(3, dtype=torch.int64, device="cuda")
    ok = {"x": x, "table": table, "positions": at}
    for name, bad in (("x", x[0]), ("x", x.transpose(1, 2)), ("table", table[0]), ("table", table[:, ::2]), ("table", table.cpu()),
                      ("positions", at[:2]), ("positions", at.cpu()), ("out", x[:2]), ("out", x[:, :3])):
        with pytest.raises(ValueError, match=name):
            capi.rotary_apply(**{**ok, name: bad})
    for name, bad in (("x", x.float()), ("table", table.double()), ("positions", at.int()), ("out", x.half())):
        with pytest.raises(TypeError, match=name):
            capi.rotary_apply(**{**ok, name: bad})
    with pytest.raises(capi.I8qlError):  # a token without a row
        capi.rotary_apply(x, table[:2])
    f = torch.ones(4, dtype=torch.float64, device="cuda")
    for bad in (dict(freqs=f[None]), dict(freqs=f[::2]), dict(positions=-1), dict(positions=at[None]), dict(table=table)):
        with pytest.raises(ValueError):
            capi.rotary_table(**{"freqs": f, "positions": at, **bad})
    codes, params = capi.kv_cache_alloc(2, 4, 16, 64)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda") - 1
    ok = {"q": x, "k": x, "v": x, "table": table, "slots": slots, "codes": codes, "params": params, "positions": at}
    for bad in (dict(q=None, q_out=x), dict(v=x[:2]), dict(q=x[:2]), dict(q_out=x[:2]), dict(slots=slots[:2]), dict(k=x[:, :2]),
                dict(table=table[None]), dict(positions=at[:1]), dict(q=x[..., :32])):
        with pytest.raises(ValueError):
            capi.kv_cache_store_rotary(**{**ok, **bad})
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
