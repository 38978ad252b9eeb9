"""How far a value read back from the quantized cache lies from the value
written, on the CPU from the oracle (the kernels are equal to it bit for bit).

low + scale * code is within half a scale of x, up to the fp32 roundings of
x - low and of the quotient.  The value read back is that rounded to bf16, and
as x is a bf16 value itself, the nearest bf16 is no further from low + scale *
code than x is: at most the same again, a whole scale."""

from __future__ import annotations

import numpy as np
import pytest
import torch

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
