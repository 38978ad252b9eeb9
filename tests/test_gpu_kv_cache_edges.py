"""GPU tests of attention over the quantized cache where its parts meet: row
blocks of different heights in one block's range, values that must not reach
other rows, magnitudes far apart.  Bounds: tests/kv_reference.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import capi
from tests.kv_reference import check
from tests.test_gpu_kv_cache import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    from int8_quantized_linear_gb300 import build
    build.build()
    capi.lib()
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    yield
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


def rescale(p, factor):
    """Multiplies keys and values of every sequence by powers of two: factor(b, kv, tokens) -> exponents."""
    for b, (c, s, low) in enumerate(p.seqs):
        n = p.lens[b]
        if not n:
            continue
        f = np.stack([np.exp2(factor(b, kv, np.arange(n))) for kv in (0, 1)]).astype(np.float32)[:, :, None]
        p.seqs[b] = (c, s * f, low * f)
        pages = -(-n // p.page)
        full = torch.ones((2, pages * p.page))
        full[:, :n] = torch.from_numpy(f[..., 0])
        at = p.table[b, :pages].long()
        p.params[at] = (p.params[at].float() * full.view(2, pages, 1, p.page, 1).transpose(0, 1).cuda()).to(torch.bfloat16)


@pytest.mark.parametrize("bits,d", [(4, 128), (8, 64)])
def test_low_row_blocks_between_high_ones(bits, d):
    """Blocks of at most 128 rows leave the second M tile out, blocks of more take it back in; both walk many tiles, of
    exponents that differ from tile to tile."""
    lens = [1500, 1300] * 40
    p = Problem(lens, [50, 9] * 40, 8, 2, d, bits, 16, 7 + bits, spread=0.5)
    rescale(p, lambda b, kv, j: (j // 128 * (3 + b + kv)) % 5 - 2)
    y = p.run()
    check(p, y)
    for _ in range(5):
        assert torch.equal(p.run(), y)


NON_FINITE = [("scale", float("nan")), ("low", float("nan")), ("scale", float("inf")), ("low", float("-inf"))]


@pytest.mark.parametrize("which,value", NON_FINITE)
@pytest.mark.parametrize("lens,nqs,window", [([500, 70], [3, 1], 0), ([500, 70], [60, 1], 0), ([700, 130], [200, 90], 40),
                                             ([5003, 900], [40, 70], 0)])
@pytest.mark.parametrize("bits,d", [(4, 128), (8, 128), (4, 64), (8, 64)])
def test_non_finite_rows_reach_only_rows_that_see_them(bits, d, lens, nqs, window, which, value):
    """A token whose params are not finite, among the query tokens: rows that do not see it give the bits they give
    when its params are zero, in few rows as in many; rows that see such a value are not a number."""
    p = Problem(lens, nqs, 8, 2, d, bits, 16, 40 + bits)
    first = lens[0] - nqs[0]
    bad = [first + 1, first + nqs[0] // 2, lens[0] - 1]
    at = [(int(p.table[0, t // 16]), t % 16) for t in bad]
    sees = torch.zeros(p.q.shape[0], dtype=torch.bool)
    for i in range(nqs[0]):
        sees[i] = any(t <= first + i and (not window or t > first + i - window) for t in bad)
    assert sees.any() and not sees.all()
    for kv in (0, 1):
        keep = p.params.clone()
        for page, off in at:
            p.params[page, kv, 1, off] = 0.0
        want = p.run(window=window)
        for page, off in at:
            p.params[page, kv, 1, off, 0 if which == "scale" else 1] = value
        y = p.run(window=window)
        p.params = keep
        assert torch.equal(y[:, :4], want[:, :4])          # the other cache head
        assert torch.equal(y[~sees, 4:], want[~sees, 4:])  # rows that see none of them
        if kv == 1:
            assert torch.isnan(y[sees, 4:]).any(-1).all() or value in (float("inf"), float("-inf"))
            assert not torch.isfinite(y[sees, 4:]).all(-1).any()


@pytest.mark.parametrize("nq", [1, 4, 60, 200])
@pytest.mark.parametrize("far", [16, 20, 22, 25, 28, 31, 40])
@pytest.mark.parametrize("bits,d", [(4, 128), (8, 64)])
def test_logits_of_any_size(bits, d, far, nq):
    """Keys 2^far times the queries' size: logits whose fp32 spacing passes the softmax's own units."""
    p = Problem([700, 130], [nq, 1], 8, 2, d, bits, 16, 60 + far)
    rescale(p, lambda b, kv, j: np.where(kv == 0, far, 0) + 0 * j)
    y = p.run()
    # (a row is pinned where its largest logits lie further apart than they may be off: nearly all)
    assert check(p, y) > 0.9


FAR = [(nq, 0, far) for nq in (3, 150) for far in (12, 16, 20, 24, 30)] + [(3, 1, 8), (3, 1, 12)] + [
    (150, 1, far) for far in (8, 12, 16, 20, 24, 30)]


@pytest.mark.parametrize("nq,kv,far", FAR)
@pytest.mark.parametrize("bits,d", [(4, 128), (8, 128), (4, 64), (8, 64)])
def test_a_token_far_larger_than_its_neighbours(bits, d, nq, kv, far):
    """A key (or value) 2^far times the rest of its tile, hidden from most rows or outweighed by its strongly negative
    logit: the small tokens decide those outputs.  (Few rows hold value scales in fp16 relative to the largest: less
    far.)"""
    p = Problem([700], [nq], 8, 2, d, bits, 16, far + bits)
    big = [600, 640, 698]
    if kv == 0:  # key channels of the big tokens all of one sign, against the queries' sign: far below every other logit
        p.q = p.q.abs()
        c, s, low = p.seqs[0]
        for t in big:
            low[0, t] = -np.abs(low[0, t]) - s[0, t] * 2 ** bits
            page, off = int(p.table[0, t // 16]), t % 16
            p.params[page, 0, :, off, 1] = torch.from_numpy(low[0, t]).to(torch.bfloat16).cuda()
            low[0, t] = p.params[page, 0, :, off, 1].float().cpu().numpy()
    rescale(p, lambda b, x, j: np.where(np.isin(j, big) & (x == kv), far, 0))
    assert check(p, p.run()) > 0.9


class Elsewhere(torch.Tensor):
    """A tensor that says it is on another device (its memory is never touched there)."""

    def get_device(self):
        return 1

    @property
    def device(self):
        return torch.device("cuda:1")


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Pointers of one device handed to a kernel on another would fault where the two do not share memory."""
    p = Problem([50, 20], [2, 1], 4, 2, 64, 4, 16, 3)
    k, slots, q = torch.zeros((5, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.arange(5, device="cuda"), p.q.cuda()
    calls = {
        "store": (lambda **a: capi.kv_cache_store(a["k"], a["v"], a["slots"], a["codes"], a["params"]),
                  dict(k=k, v=k.clone(), slots=slots, codes=p.codes, params=p.params)),
        "load": (lambda **a: capi.kv_cache_load(a["codes"], a["params"], a["slots"], 64, k=a["k"], v=a["v"]),
                 dict(k=k.clone(), v=k.clone(), slots=slots, codes=p.codes, params=p.params)),
        "attention": (lambda **a: capi.kv_cache_attention(a["q"], a["codes"], a["params"], a["page_table"], a["kv_lens"],
                                                          q_offsets=a["q_offsets"], out=a["out"], workspace=a["workspace"]),
                      dict(q=q, codes=p.codes, params=p.params, page_table=p.table, kv_lens=p.kv_lens, q_offsets=p.offsets,
                           out=torch.zeros_like(q), workspace=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))),
    }

    class Fake:  # of the library: nothing may reach it
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    for call, args in calls.values():
        call(**args)
        torch.cuda.synchronize()
        with monkeypatch.context() as m:
            m.setattr(capi, "lib", Fake)
            for name in args:
                with pytest.raises(ValueError, match=f"{name} .*device"):
                    call(**{**args, name: args[name].as_subclass(Elsewhere)})
            m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
            with pytest.raises(ValueError, match="codes .*device"):
                call(**args)
