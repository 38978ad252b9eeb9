"""Host checks of the quantized key/value cache: refusals of the C ABI and of
the binding, the oracle's quantization pinned by hand, and the oracle's
attention against a plain softmax and its own properties (no GPU)."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import build as lib_build
from int8_quantized_linear_gb300 import capi
from oracle import kv_cache as oracle

A, B, C, D, E = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return capi.lib()


def _with(ok, **changes):
    args = list(ok)
    for i, v in changes.items():
        args[int(i[1:])] = v
    return args


INVALID, UNSUPPORTED = capi.I8QL_ERR_INVALID_ARG, capi.I8QL_ERR_UNSUPPORTED


def test_store_refusals(lib):
    f = lib.kv_cache_store
    #     k  v  k_stride v_stride slots codes params T H D bits page pages stream
    ok = (A, B, 1024, 1024, C, D, E, 8, 8, 128, 4, 64, 10, None)
    assert f(*_with(ok, _9=96)) == UNSUPPORTED
    assert f(*_with(ok, _10=2)) == UNSUPPORTED
    assert f(*_with(ok, _11=48)) == UNSUPPORTED           # not a power of two
    assert f(*_with(ok, _11=8)) == UNSUPPORTED
    assert f(*_with(ok, _11=512)) == UNSUPPORTED
    assert f(*_with(ok, _7=1 << 27)) == UNSUPPORTED       # T * H
    assert f(*_with(ok, _12=1 << 31)) == UNSUPPORTED
    for i in (8, 9, 11, 12):
        assert f(*_with(ok, **{f"_{i}": 0})) == INVALID
    assert f(*_with(ok, _7=-1)) == INVALID
    assert f(*_with(ok, _2=1016)) == INVALID              # tokens would overlap
    assert f(*_with(ok, _3=1028)) == INVALID              # stride % 8
    for i, off in ((0, 8), (1, 8), (4, 4), (5, 8), (6, 8)):
        assert f(*_with(ok, **{f"_{i}": ok[i] + off})) == INVALID
        assert f(*_with(ok, **{f"_{i}": None})) == INVALID
    assert f(*_with(ok, _7=0, _0=None, _1=None, _4=None, _5=None, _6=None)) == capi.I8QL_OK
    if not torch.cuda.is_available():
        assert f(*ok) == capi.I8QL_ERR_NO_DEVICE


def test_load_refusals(lib):
    f = lib.kv_cache_load
    #     codes params slots k v T H D bits page pages stream
    ok = (A, B, C, D, E, 8, 8, 64, 8, 16, 10, None)
    assert f(*_with(ok, _7=32)) == UNSUPPORTED
    assert f(*_with(ok, _8=3)) == UNSUPPORTED
    assert f(*_with(ok, _9=33)) == UNSUPPORTED
    assert f(*_with(ok, _6=0)) == INVALID
    for i in range(5):
        assert f(*_with(ok, **{f"_{i}": None})) == INVALID
        assert f(*_with(ok, **{f"_{i}": ok[i] + 4})) == INVALID
    assert f(*_with(ok, _5=0)) == capi.I8QL_OK


def test_attention_refusals(lib):
    f = lib.kv_cache_attention
    #     q q_stride codes params table width lens offsets out B T Hq H D bits page pages max_q window scale ws bytes stream
    ok = (A, 4096, B, C, D, 16, E, None, A, 4, 4, 32, 8, 128, 4, 64, 100, 1, 0, 0.1, A, 1 << 30, None)
    assert f(*_with(ok, _13=256)) == UNSUPPORTED
    assert f(*_with(ok, _14=16)) == UNSUPPORTED
    assert f(*_with(ok, _15=40)) == UNSUPPORTED
    assert f(*_with(ok, _5=(1 << 31) // 64)) == UNSUPPORTED  # positions leave 31 bits
    assert f(*_with(ok, _7=E, _10=1 << 28)) == UNSUPPORTED   # rows of a head group leave 30 bits
    assert f(*_with(ok, _12=7)) == INVALID                 # query heads not a multiple of the cache's
    assert f(*_with(ok, _10=5)) == INVALID                 # one token per sequence without offsets
    assert f(*_with(ok, _1=4088)) == INVALID
    assert f(*_with(ok, _1=4100)) == INVALID
    assert f(*_with(ok, _18=-1)) == INVALID
    assert f(*_with(ok, _19=float("nan"))) == INVALID
    assert f(*_with(ok, _19=float("inf"))) == INVALID
    assert f(*_with(ok, _19=3e38)) == INVALID              # times log2 e leaves fp32
    for i in (5, 11, 12, 17):
        assert f(*_with(ok, **{f"_{i}": 0})) == INVALID
    assert f(*_with(ok, _9=0, _7=E)) == INVALID            # query tokens of no sequence
    for i, off in ((0, 8), (2, 8), (3, 8), (4, 2), (6, 2), (8, 8)):
        assert f(*_with(ok, **{f"_{i}": None})) == INVALID
        assert f(*_with(ok, **{f"_{i}": ok[i] + off})) == INVALID
    assert f(*_with(ok, _7=E + 2)) == INVALID
    assert f(*_with(ok, _9=0, _10=0)) == capi.I8QL_OK
    if not torch.cuda.is_available():
        assert f(*ok) == capi.I8QL_ERR_NO_DEVICE
    n = ctypes.c_int64(-1)
    w = lib.i8ql_kv_attention_workspace
    assert w(4, 4, 32, 8, 128, 4, 64, 16, 1, None) == INVALID
    assert w(4, 4, 32, 8, 96, 4, 64, 16, 1, ctypes.byref(n)) == UNSUPPORTED
    assert w(4, 4, 32, 5, 128, 4, 64, 16, 1, ctypes.byref(n)) == INVALID
    assert w(0, 0, 32, 8, 128, 4, 64, 16, 1, ctypes.byref(n)) == capi.I8QL_OK and n.value == 0


def test_binding_refusals(lib):
    codes, params = capi.kv_cache_alloc(3, 2, 16, 64, bits=4, device="cpu")
    assert tuple(codes.shape) == (3, 2, 2, 16, 32) and tuple(params.shape) == (3, 2, 2, 16, 2)
    with pytest.raises(ValueError):
        capi.kv_cache_alloc(3, 2, 16, 64, bits=5)
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        capi.kv_cache_store(k, k, slots, codes, params)
    with pytest.raises(ValueError, match="codes"):
        capi.kv_cache_store(k[..., :32], k[..., :32], slots, codes[..., :20], params)
    with pytest.raises(ValueError, match="codes"):
        capi.kv_cache_load(codes[:, 0], params, slots, 64)
    with pytest.raises(TypeError):
        capi.kv_cache_load(codes.to(torch.int8), params, slots, 64)


def test_status_strings():
    assert "slot" in capi.status_string(capi.I8QL_ERR_BAD_INDEX)
    assert capi.status_string(9) == "unknown status"


# ------------------------------------------------------------------ the oracle

def test_oracle_quantizes_by_hand():
    # range 15 at 4 bits: scale exactly 1, codes are the values above the lowest, ties to even
    row = np.full(64, -5.0, np.float32)
    row[:6] = [10.0, -4.5, -3.5, -2.5, 0.25, 9.75]
    c, s, low = oracle.quantize(row, 4)
    assert s == 1.0 and low == -5.0
    assert c[:6].tolist() == [15, 0, 2, 2, 5, 15]
    # range 1: 1/15 lies between two bf16; the scale is the upper one, and the top value keeps a code in range
    c, s, low = oracle.quantize(np.array([0.0, 1.0] * 32, np.float32), 4)
    assert s == np.array([0x3D89 << 16], np.uint32).view(np.float32)[0]
    assert s >= np.float32(1) / 15 and c.max() == 15
    # a constant row: scale 0, low the value
    c, s, low = oracle.quantize(np.full(64, 3.25, np.float32), 8)
    assert s == 0 and low == 3.25 and not c.any()
    # the smallest subnormal difference still has a scale above zero
    tiny = np.zeros(64, np.float32)
    tiny[0] = np.array([1 << 16], np.uint32).view(np.float32)[0]
    c, s, _ = oracle.quantize(tiny, 4)
    assert s > 0 and c[0] > 0 and not c[1:].any()


@pytest.mark.parametrize("bits", [4, 8])
def test_oracle_round_trip_is_within_half_a_step(bits):
    rng = np.random.default_rng(bits)
    x = torch.from_numpy(rng.standard_normal((200, 128)) * 10.0 ** rng.integers(-6, 6, (200, 1))).to(torch.bfloat16)
    x = x.double().numpy()
    c, s, low = oracle.quantize(x, bits)
    err = np.abs(oracle.values(c, s, low) - x)
    # half a step, and the fp32 roundings of x - low and of the quotient
    assert np.all(err <= s[:, None] * (0.5 + 2.0 ** -14))
    assert np.array_equal(oracle.unpack(oracle.pack(c, bits), bits), c)


def test_oracle_attention_is_a_softmax_average():
    rng = np.random.default_rng(3)
    n, h, d, nq = 9, 2, 64, 3
    codes = rng.integers(0, 16, (2, n, h, d)).astype(np.uint8)
    scale = np.full((2, n, h), 0.25, np.float32)
    low = np.full((2, n, h), -2.0, np.float32)
    q = rng.standard_normal((nq, 2 * h, d))
    kv = torch.from_numpy(oracle.values(codes, scale, low))
    got = oracle.attention(q, codes, scale, low, nq, 0, 0.125).out
    mask = torch.arange(n) <= torch.arange(n - nq, n)[:, None]
    x = torch.einsum("qhd,khd->hqk", torch.from_numpy(q), kv[0].repeat_interleave(2, 1)) * 0.125
    p = torch.softmax(x.masked_fill(~mask, float("-inf")), -1)
    ref = torch.einsum("hqk,khd->qhd", p, kv[1].repeat_interleave(2, 1)).numpy()
    assert np.allclose(got, ref, rtol=1e-12, atol=1e-14)
    # a window of one token: its own value
    one = oracle.attention(q, codes, scale, low, nq, 1, 0.125).out
    assert np.allclose(one, kv[1][n - nq:].repeat_interleave(2, 1).numpy(), rtol=0, atol=1e-15)
    # more queries than tokens: the first ones see nothing
    none = oracle.attention(np.ones((4, 2 * h, d)), codes[:, :2], scale[:, :2], low[:, :2], 4, 0, 0.125).out
    assert not none[:2].any() and none[2:].any()
