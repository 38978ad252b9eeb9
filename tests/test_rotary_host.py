"""Host checks of rotary positions: refusals of the C ABI and of the binding,
the frequencies and their scalings, the oracle against complex products."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import build as lib_build
from int8_quantized_linear_gb300 import capi
from oracle import rotary as oracle

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


def test_table_refusals(lib):
    f = lib.rotary_table
    #     freqs positions table P F amplitude stream
    ok = (A, B, C, 100, 64, 1.0, None)
    assert f(*_with(ok, _4=0)) == INVALID
    assert f(*_with(ok, _4=capi.I8QL_ROTARY_MAX_D // 2 + 1)) == UNSUPPORTED
    assert f(*_with(ok, _3=-1)) == INVALID
    assert f(*_with(ok, _3=1 << 31)) == UNSUPPORTED
    assert f(*_with(ok, _5=float("nan"))) == INVALID
    assert f(*_with(ok, _5=float("inf"))) == INVALID
    assert f(*_with(ok, _0=None)) == INVALID
    assert f(*_with(ok, _0=A + 4)) == INVALID
    assert f(*_with(ok, _1=B + 4)) == INVALID
    assert f(*_with(ok, _2=None)) == INVALID
    assert f(*_with(ok, _2=C + 8)) == INVALID
    assert f(*_with(ok, _0=None, _1=None, _2=None, _3=0)) == capi.I8QL_OK
    if not torch.cuda.is_available():
        assert f(*ok) == capi.I8QL_ERR_NO_DEVICE


def test_apply_refusals(lib):
    f = lib.rotary_apply
    #     x x_stride table rows positions out out_stride T heads D rot interleaved backward stream
    ok = (A, 1024, B, 100, C, D, 1024, 10, 8, 128, 128, 0, 0, None)
    assert f(*_with(ok, _9=132)) == UNSUPPORTED
    assert f(*_with(ok, _9=capi.I8QL_ROTARY_MAX_D + 8, _1=8192, _6=8192)) == UNSUPPORTED
    assert f(*_with(ok, _10=136)) == UNSUPPORTED                    # more than D
    assert f(*_with(ok, _10=20)) == UNSUPPORTED
    assert f(*_with(ok, _3=1 << 31)) == UNSUPPORTED
    assert f(*_with(ok, _7=1 << 28)) == UNSUPPORTED                 # T * heads
    assert f(*_with(ok, _8=65536, _1=1 << 24, _6=1 << 24)) == UNSUPPORTED
    for i in (8, 9, 10):
        assert f(*_with(ok, **{f"_{i}": 0})) == INVALID
    assert f(*_with(ok, _3=-1)) == INVALID
    assert f(*_with(ok, _7=-1)) == INVALID
    assert f(*_with(ok, _11=2)) == INVALID
    assert f(*_with(ok, _12=-1)) == INVALID
    assert f(*_with(ok, _4=None, _3=9)) == INVALID                  # a row for each token
    for i, off in ((0, 8), (2, 8), (4, 4), (5, 8)):
        assert f(*_with(ok, **{f"_{i}": ok[i] + off})) == INVALID
    for i in (0, 2, 5):
        assert f(*_with(ok, **{f"_{i}": None})) == INVALID
    for i in (1, 6):
        assert f(*_with(ok, **{f"_{i}": 1016})) == INVALID          # tokens would overlap
        assert f(*_with(ok, **{f"_{i}": 1028})) == INVALID          # stride % 8
    assert f(*_with(ok, _7=0, _0=None, _2=None, _4=None, _5=None)) == capi.I8QL_OK
    # rows that are partly the same: refused, unless they are the very same
    assert f(*_with(ok, _5=A, _6=1032)) == INVALID
    assert f(*_with(ok, _5=A + 16)) == INVALID
    assert f(*_with(ok, _0=A + 16, _5=A)) == INVALID
    assert f(*_with(ok, _5=A + 2 * 2048, _1=2048, _6=1024)) == INVALID
    assert f(*_with(ok, _5=A + 2 * 1016, _1=2048, _6=2048)) == INVALID
    if not torch.cuda.is_available():
        nothing = capi.I8QL_ERR_NO_DEVICE
        assert f(*ok) == nothing
        assert f(*_with(ok, _5=A)) == nothing
        assert f(*_with(ok, _5=A + 2 * 1024, _1=2048, _6=2048)) == nothing  # neighbours in the same rows
        assert f(*_with(ok, _5=A, _6=1032, _7=1)) == nothing                # one token: strides do not matter


def test_store_rotary_refusals(lib):
    f = lib.kv_cache_store_rotary
    #     q q_stride q_out q_out_stride k v k_stride v_stride table rows positions slots codes params
    #     T Hq H D bits page pages rot interleaved stream
    ok = (A, 4096, B, 4096, C, D, 1024, 1024, E, 100, F, A, B, C, 10, 32, 8, 128, 4, 64, 10, 128, 0, None)
    assert f(*_with(ok, _17=96)) == UNSUPPORTED
    assert f(*_with(ok, _18=2)) == UNSUPPORTED
    assert f(*_with(ok, _19=48)) == UNSUPPORTED
    assert f(*_with(ok, _21=8)) == UNSUPPORTED
    assert f(*_with(ok, _21=144)) == UNSUPPORTED
    assert f(*_with(ok, _14=1 << 26)) == UNSUPPORTED
    assert f(*_with(ok, _15=65536)) == UNSUPPORTED
    assert f(*_with(ok, _15=-1)) == INVALID
    for i in (16, 17, 19, 20, 21):
        assert f(*_with(ok, **{f"_{i}": 0})) == INVALID
    assert f(*_with(ok, _22=3)) == INVALID
    assert f(*_with(ok, _10=None, _9=9)) == INVALID
    for i in (0, 2, 4, 5, 8, 11, 12, 13):
        assert f(*_with(ok, **{f"_{i}": None})) == INVALID
        assert f(*_with(ok, **{f"_{i}": ok[i] + 4})) == INVALID
    for i in (1, 3, 6, 7):
        assert f(*_with(ok, **{f"_{i}": ok[i] - 8})) == INVALID
    assert f(*_with(ok, _2=A + 16)) == INVALID
    assert f(*_with(ok, _14=0)) == capi.I8QL_OK
    if not torch.cuda.is_available():
        assert f(*ok) == capi.I8QL_ERR_NO_DEVICE
        assert f(*_with(ok, _0=None, _2=None, _15=0)) == capi.I8QL_ERR_NO_DEVICE  # no queries


def test_store_rotary_refuses_queries_over_keys(lib):
    f = lib.kv_cache_store_rotary
    # a fused projection of 32 + 8 + 8 heads of 128 channels
    q, k, v, step = A, A + 2 * 4096, A + 2 * 5120, 6144
    ok = (q, step, q, step, k, v, step, step, E, 100, F, B, C, D, 10, 32, 8, 128, 4, 64, 10, 128, 0, None)
    for i in (4, 5):
        assert f(*_with(ok, _2=B, _3=4096, **{f"_{i}": B + 2 * 4096})) == INVALID    # over the second row
        assert f(*_with(ok, **{f"_{i}": A})) == INVALID
        assert f(*_with(ok, **{f"_{i}": A + 2 * 4088})) == INVALID
        assert f(*_with(ok, **{f"_{i}": A + 2 * (step + 4088)})) == INVALID
        assert f(*_with(ok, _2=A + 2 * 8, **{f"_{i}": A})) == INVALID
    if not torch.cuda.is_available():
        nothing = capi.I8QL_ERR_NO_DEVICE
        assert f(*ok) == nothing                      # in place, beside the keys
        assert f(*_with(ok, _4=v, _5=k)) == nothing


def test_binding_refusals(lib):
    x, table = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((10, 64))
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        capi.rotary_apply(x, table)
    with pytest.raises(ValueError, match="x must be"):
        capi.rotary_apply(x[0], table)
    with pytest.raises(TypeError, match="freqs"):
        capi.rotary_table(torch.zeros(4), 10)
    with pytest.raises(ValueError, match="freqs must be a CUDA tensor"):
        capi.rotary_table(torch.zeros(4, dtype=torch.float64), 10)


def test_frequencies():
    f = capi.rotary_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    assert f[0] == 1.0 and math.isclose(float(f[16]), 0.01, rel_tol=1e-14)
    assert torch.equal(capi.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu") * 4, f)
    g = capi.rotary_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert g[0] == f[0] and math.isclose(float(f[-1] / g[-1]), 4.0, rel_tol=1e-12)
    for kind in ("turns", "index"):
        g = capi.rotary_frequencies(128, 1e6, kind, 8.0, original=4096, low=1.0, high=32.0, device="cpu")
        f = capi.rotary_frequencies(128, 1e6, device="cpu")
        turns, ratio = 4096 * f / (2 * math.pi), f / g
        assert torch.equal(g[turns >= 32 * 1.5], f[turns >= 32 * 1.5])
        assert torch.allclose(ratio[turns <= 1 / 1.5], torch.tensor(8.0, dtype=torch.float64), rtol=1e-12)
        assert (ratio[1:] >= ratio[:-1] - 1e-12).all() and ((ratio > 1.01) & (ratio < 7.99)).any()
    for bad in (dict(rot=63), dict(rot=0), dict(base=1.0), dict(factor=0.5), dict(scaling="other"), dict(scaling="turns"),
                dict(scaling="index", original=100, low=2.0, high=1.0), dict(rot=2, scaling="base")):
        with pytest.raises(ValueError):
            capi.rotary_frequencies(**{"rot": 64, "device": "cpu", **bad})


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, angle = rng.standard_normal((5, 3, 40)), rng.standard_normal((5, 16)) * 10
    y = oracle.turn64(x, np.concatenate([np.cos(angle), np.sin(angle)], 1), interleaved)
    pick = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    z = (x[..., pick[0]] + 1j * x[..., pick[1]]) * np.exp(1j * angle)[:, None]
    assert np.allclose(y[..., pick[0]], z.real) and np.allclose(y[..., pick[1]], z.imag)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    back = oracle.turn64(y, np.concatenate([np.cos(angle), np.sin(angle)], 1), interleaved, True)
    assert np.allclose(back, x)


def test_oracle_table_of_far_positions():
    f = np.array([1.0, 0.3, 1e-5])
    at = [0, 1, -7, 10 ** 6]
    want = np.concatenate([np.cos(np.outer(at, f)), np.sin(np.outer(at, f))], 1)
    assert np.allclose(oracle.table(f, at), want, atol=1e-9)
