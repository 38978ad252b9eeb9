"""Host checks of frequencies blended by index (rotary_frequencies, "index"),
where the blend ends inside the pairs and behind the last one."""

from __future__ import annotations

import math

import pytest
import torch

from int8_quantized_linear_gb300 import capi


@pytest.mark.parametrize("rot,base,original,low,high,factor", [
    (128, 1e6, 4096, 1.0, 32.0, 8.0),       # ends inside
    (128, 1e4, 4096, 1.0, 32.0, 4.0),
    (128, 1e4, 65536, 1.0, 32.0, 4.0),      # the last pair turns more than `low` times
    (128, 1e4, 131072, 1.0, 32.0, 4.0),
    (64, 1e4, 131072, 1.0, 4.0, 16.0),
    (64, 500.0, 8192, 1.0, 32.0, 2.0),
    (32, 100.0, 1 << 20, 1.0, 2.0, 4.0),    # all pairs turn more than `high` times: none is changed
])
def test_blend_by_index(rot, base, original, low, high, factor):
    n = rot // 2
    f = capi.rotary_frequencies(rot, base, device="cpu")
    got = capi.rotary_frequencies(rot, base, "index", factor, original=original, low=low, high=high, device="cpu")
    # the index x (not whole) at which a pair turns t times: original base^(-x / n) / 2 pi = t
    index = lambda t: n * math.log(original / (2 * math.pi * t), base)  # noqa: E731
    begin, end = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
    for i in range(n):
        keep = 1.0 if i <= begin else max(1.0 - (i - begin) / (end - begin), 0.0)
        want = float(f[i]) * (keep + (1.0 - keep) / factor)
        assert math.isclose(float(got[i]), want, rel_tol=1e-12), (i, begin, end)
        turns = original * float(f[i]) / (2 * math.pi)
        if turns >= high:  # as it is, but for the rounding of the indices to whole ones
            assert float(got[i]) >= float(f[i]) * (1 - 1.0 / max(end - begin, 1))
        if turns > low and begin < i < end:
            assert float(f[i]) / factor < float(got[i]) < float(f[i])


def test_the_last_pair_is_blended_in_part():
    """131072 positions, base 1e4: the last of 64 pairs turns 2.4 times, and a single turn would be at index 69.1."""
    f = capi.rotary_frequencies(128, 1e4, device="cpu")
    got = capi.rotary_frequencies(128, 1e4, "index", 4.0, original=131072, high=32.0, device="cpu")
    assert 2.4 < 131072 * float(f[63]) / (2 * math.pi) < 2.42
    keep = 1 - (63 - 45) / (70 - 45)
    assert math.isclose(float(got[63] / f[63]), keep + (1 - keep) / 4, rel_tol=1e-12)
    assert torch.equal(got[:46], f[:46])
