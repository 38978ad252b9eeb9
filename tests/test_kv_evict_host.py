"""Host checks of cache eviction: refusals of the C ABI and of the binding, and
the oracle against hand-made cases and a plain softmax."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import build as lib_build
from int8_quantized_linear_gb300 import capi
from oracle import kv_cache as cache_oracle
from oracle import kv_evict as oracle

A, B, C, D, E, F = (0x100000 * i for i in range(1, 7))  # never dereferenced
INVALID, UNSUPPORTED = capi.I8QL_ERR_INVALID_ARG, capi.I8QL_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return capi.lib()


def _with(ok, **changes):
    args = list(ok)
    for i, v in changes.items():
        args[int(i[1:])] = v
    return args


def test_weights_refusals(lib):
    f = lib.kv_cache_weights
    #     q q_stride codes params table width lens offsets previous weights B T Hq H D bits page pages max_q window
    #     scale workspace bytes stream
    ok = (A, 4096, B, C, D, 16, E, None, None, F, 4, 4, 32, 8, 128, 4, 64, 100, 1, 0, 0.1, A, 1 << 40, None)
    assert f(*_with(ok, _14=256)) == UNSUPPORTED
    assert f(*_with(ok, _15=16)) == UNSUPPORTED
    assert f(*_with(ok, _16=40)) == UNSUPPORTED
    assert f(*_with(ok, _5=1 << 40)) == UNSUPPORTED
    assert f(*_with(ok, _10=1 << 31)) == UNSUPPORTED
    assert f(*_with(ok, _12=65536, _1=1 << 24)) == UNSUPPORTED
    for i in (5, 12, 13, 14, 16, 17, 18):
        assert f(*_with(ok, **{f"_{i}": 0})) == INVALID
    assert f(*_with(ok, _12=33)) == INVALID
    assert f(*_with(ok, _19=-1)) == INVALID
    assert f(*_with(ok, _20=float("nan"))) == INVALID
    assert f(*_with(ok, _11=5)) == INVALID                # one query each without offsets
    assert f(*_with(ok, _1=4088)) == INVALID
    assert f(*_with(ok, _7=E + 2)) == INVALID
    assert f(*_with(ok, _8=E + 4)) == INVALID
    for i, off in ((0, 8), (2, 8), (3, 8), (4, 2), (6, 2), (9, 8)):
        assert f(*_with(ok, **{f"_{i}": ok[i] + off})) == INVALID
        assert f(*_with(ok, **{f"_{i}": None})) == INVALID
    assert f(*_with(ok, _10=0, _11=0)) == capi.I8QL_OK
    assert f(*_with(ok, _10=0, _7=E)) == INVALID          # queries without a sequence
    if not torch.cuda.is_available():
        assert f(*ok) == capi.I8QL_ERR_NO_DEVICE
    n = ctypes.c_int64(-1)
    g = lib.i8ql_kv_weights_workspace
    assert g(4, 4, 33, 8, 128, 4, 64, 16, 1, ctypes.byref(n)) == INVALID
    assert g(4, 4, 32, 8, 128, 4, 64, 16, 1, None) == INVALID
    assert g(4, 4, 32, 8, 100, 4, 64, 16, 1, ctypes.byref(n)) == UNSUPPORTED
    assert g(4, 0, 32, 8, 128, 4, 64, 16, 0, ctypes.byref(n)) == capi.I8QL_OK and n.value == 0


def test_weights_refuse_overlapping_buffers(lib):
    f = lib.kv_cache_weights
    previous, size = F, 100 * 8 * 64 * 4
    ok = (A, 4096, B, C, D, 16, E, None, previous, F, 4, 4, 32, 8, 128, 4, 64, 100, 1, 0, 0.1, A, 1 << 40, None)
    for off in (16, size - 16):
        assert f(*_with(ok, _9=F + off)) == INVALID
        assert f(*_with(ok, _8=F + off)) == INVALID
    if not torch.cuda.is_available():
        for off in (0, size):
            assert f(*_with(ok, _9=F + off)) == capi.I8QL_ERR_NO_DEVICE


def test_evict_refusals(lib):
    f = lib.kv_cache_evict
    #     codes params weights table width lens new_table new_width new_lens kept B H D bits page pages budget first last stream
    ok = (A, B, C, D, 16, E, F, 8, E + 4096, E + 8192, 4, 8, 128, 4, 64, 100, 256, 4, 100, None)
    assert f(*_with(ok, _12=96)) == UNSUPPORTED
    assert f(*_with(ok, _13=5)) == UNSUPPORTED
    assert f(*_with(ok, _14=8)) == UNSUPPORTED
    assert f(*_with(ok, _10=1 << 31)) == UNSUPPORTED
    assert f(*_with(ok, _4=1 << 40)) == UNSUPPORTED
    assert f(*_with(ok, _7=1 << 40)) == UNSUPPORTED
    assert f(*_with(ok, _16=1 << 32)) == UNSUPPORTED
    assert f(*_with(ok, _16=1 << 28, _10=64)) == UNSUPPORTED     # B * H * budget
    for i in (4, 7, 11, 12, 14, 15, 16):
        assert f(*_with(ok, **{f"_{i}": 0})) == INVALID
    for i in (10, 17, 18):
        assert f(*_with(ok, **{f"_{i}": -1})) == INVALID
    assert f(*_with(ok, _17=157)) == INVALID                     # first + last > budget
    assert f(*_with(ok, _17=(1 << 62), _18=(1 << 62))) == INVALID
    assert f(*_with(ok, _6=D)) == INVALID                        # in place, but another width
    assert f(*_with(ok, _8=E)) == INVALID                        # the new lengths over the old
    assert f(*_with(ok, _8=E + 12)) == INVALID
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 2), (5, 2), (6, 2), (8, 2), (9, 2)):
        assert f(*_with(ok, **{f"_{i}": ok[i] + off})) == INVALID
    for i in (0, 1, 2, 3, 5, 8, 9):
        assert f(*_with(ok, **{f"_{i}": None})) == INVALID
    assert f(*_with(ok, _10=0)) == capi.I8QL_OK
    if not torch.cuda.is_available():
        assert f(*ok) == capi.I8QL_ERR_NO_DEVICE
        assert f(*_with(ok, _6=None)) == capi.I8QL_ERR_NO_DEVICE
        assert f(*_with(ok, _6=D, _7=16)) == capi.I8QL_ERR_NO_DEVICE
        assert f(*_with(ok, _8=E + 16)) == capi.I8QL_ERR_NO_DEVICE


def test_binding_refusals(lib):
    codes, params = capi.kv_cache_alloc(6, 2, 16, 64, device="cpu")
    w = torch.zeros((6, 2, 16))
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="codes must be a CUDA tensor"):
        capi.kv_cache_weights(q, codes, params, table, lens, w)
    with pytest.raises(ValueError, match="codes must be a CUDA tensor"):
        capi.kv_cache_evict(codes, params, w, table, lens, 8)
    with pytest.raises(ValueError, match="codes must be"):
        capi.kv_cache_evict(codes[0], params, w, table, lens, 8)


def test_oracle_choice():
    w = np.array([5, 1, 9, np.nan, 9, -0.0, 0.0, 9, -np.inf, 2], np.float32)
    pick = lambda *a: oracle.choose(w, 10, *a).tolist()  # noqa: E731
    assert pick(10, 0, 0) == list(range(10)) == pick(50, 0, 0)
    assert pick(1, 0, 0) == [2]
    assert pick(2, 0, 0) == [2, 4]
    assert pick(3, 1, 1) == [0, 2, 9]
    assert pick(4, 2, 2) == [0, 1, 8, 9]
    assert pick(7, 0, 0) == [0, 1, 2, 4, 5, 7, 9]  # of -0 and 0 the first
    assert pick(9, 0, 0) == [0, 1, 2, 4, 5, 6, 7, 8, 9]


@pytest.mark.parametrize("window", [0, 5])
def test_oracle_weights(window):
    rng = np.random.default_rng(3)
    n, nq, heads, g, d = 17, 4, 2, 3, 64
    c, s, low = cache_oracle.quantize(rng.standard_normal((n, heads, d)), 4)
    q = rng.standard_normal((nq, heads * g, d))
    sums, bound, seen = oracle.weights(q, c, s, low, nq, window, 0.1, 8)
    k = torch.from_numpy(cache_oracle.values(c, s, low)).repeat_interleave(g, 1)
    x = 0.1 * torch.einsum("qhd,khd->hqk", torch.from_numpy(q), k)
    j, p = torch.arange(n), torch.arange(n - nq, n)[:, None]
    hidden = (j > p) | ((j <= p - window) if window else torch.zeros((), dtype=torch.bool))
    w = torch.softmax(x.masked_fill(hidden, float("-inf")), -1).sum(1).view(heads, g, n).sum(1).numpy()
    assert np.allclose(sums, w) and (bound < 1e-3).all() and np.isclose(sums.sum(), nq * heads * g)
    assert seen.tolist() == (~hidden).any(0).tolist()
