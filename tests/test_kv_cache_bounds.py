"""Host checks of the quantized cache at its edges: how far a value read back
lies from the value written, from the oracle (the kernels are equal to it bit
for bit), and sizes of nothing.

low + scale * code is within half a scale of x, up to the fp32 roundings of
x - low and of the quotient.  The value read back is that rounded to bf16, and
as x is a bf16 value itself, the nearest bf16 is no further from low + scale *
code than x is: at most the same again, a whole scale."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import build as lib_build
from int8_quantized_linear_gb300 import capi
from oracle import kv_cache as oracle


def rows(kind, n, d, rng):
    x = rng.standard_normal((n, d)) * 10.0 ** rng.integers(-6, 6, (n, 1))
    if kind == "offset":  # a spread far below the values
        x = 3.0 + x * 10.0 ** rng.integers(-12, 0, (n, 1))
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["normal", "offset"])
@pytest.mark.parametrize("bits", [4, 8])
def test_values_are_within_half_a_scale_and_read_back_within_one(bits, kind):
    x = rows(kind, 400, 128, np.random.default_rng(bits))
    c, s, low = oracle.quantize(x.float().numpy(), bits)
    y = oracle.values(c, s, low)
    back = torch.from_numpy(y.astype(np.float32)).to(torch.bfloat16).double().numpy()
    x = x.double().numpy()
    half = s[:, None].astype(np.float64) * (0.5 + 2.0 ** -14)
    assert np.all(np.abs(y - x) <= half)
    assert np.all(np.abs(back - x) <= 2 * half + 2.0 ** -23 * np.abs(y))
    assert np.array_equal(back.min(-1), x.min(-1))
    if bits == 8 and kind == "normal":  # half a scale would not hold
        assert (np.abs(back - x) > half).any()


def test_a_batch_without_query_tokens():
    """An upper bound of 0 query tokens is one, where there are none."""
    lib_build.build()
    #     q q_stride codes params table width lens offsets out B T Hq H D bits page pages max_q window scale ws bytes stream
    args = [0x10000, 4096, 0x20000, 0x30000, 0x40000, 16, 0x50000, 0x60000, 0x70000, 4, 0, 32, 8, 128, 4, 64, 100, 0, 0, 0.1,
            None, 0, None]
    assert capi.lib().kv_cache_attention(*args) == capi.I8QL_OK
    n = ctypes.c_int64(-1)
    assert capi.lib().i8ql_kv_attention_workspace(4, 0, 32, 8, 128, 4, 64, 16, 0, ctypes.byref(n)) == capi.I8QL_OK
    assert n.value == 0
    args[10] = 3
    assert capi.lib().kv_cache_attention(*args) == capi.I8QL_ERR_INVALID_ARG
    args[17] = -1
    assert capi.lib().kv_cache_attention(*args) == capi.I8QL_ERR_INVALID_ARG
