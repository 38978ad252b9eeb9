"""The first pass of attention weights of many query rows
(``csrc/kv_weights_many.cu``: ``add_tokens``), checked on the CPU against a
restatement of its loop in fp32.

A row's exponents are fma(x, u, -ref), where ref is a rounded number and the
product is not: the largest logit itself comes out at what ref was rounded by,
half a unit in its last place at most, and that exceeds the slack from 2^28 on.
So the loop may not go on until no exponent exceeds the slack: it takes up a
tile once more after the reference was raised, and no more.
"""

from __future__ import annotations

import numpy as np
import pytest

SLACK = np.float32(8.0)


def fma(a, b, c):
    """fp32 a b + c rounded once: the product of two fp32 numbers is exact in 64 bits, and the sum is rounded to odd
    (where it is not exact, its last bit is set) before it is rounded to fp32."""
    a, b, c = (np.float64(v) for v in (a, b, c))
    p = a * b
    s = np.asarray(p + c)
    t = s - p
    error = (p - (s - t)) + (c - t)
    s = np.where((error != 0) & (s.view(np.int64) & 1 == 0) & np.isfinite(s),
                 np.nextafter(s, np.where(error > 0, np.inf, -np.inf)), s)
    with np.errstate(over="ignore", under="ignore"):
        return s.astype(np.float32)


def add_tokens(ref, total, x, unit, most=2):
    """(reference, sum) of a row after a tile with products x; how often the tile was taken up."""
    for rounds in range(1, 60):
        shift = np.float32(0.0) if ref == -np.inf else np.float32(-ref)
        y = fma(x, unit, shift)
        again = (ref == -np.inf or y.max() > SLACK) and rounds < most
        if not again:
            with np.errstate(over="ignore"):
                return ref, np.float32(total + np.exp2(y.astype(np.float32)).sum(dtype=np.float32)), rounds
        to = np.float32(y.max() - shift)
        total = np.float32(0.0) if ref == -np.inf or total == 0 else np.float32(total * np.exp2(np.float32(ref - to)))
        ref = to
    return ref, total, rounds


def rows(far, count, seed=0):
    """Products of `count` rows with two tiles of 128 tokens, logits of some 2^far."""
    rng = np.random.default_rng(seed + far)
    unit = (rng.random(count).astype(np.float32) + np.float32(0.5)) * np.float32(2.0 ** (far - 20))
    return rng.standard_normal((count, 2, 128)).astype(np.float32) * np.float32(2.0 ** 19), unit


def test_fma_rounds_once():
    # 1 + 2^-24 + 2^-60 lies above the middle of 1 and its neighbour; 64 bits would lose the last part
    a, b = np.float32(2.0 ** -30), np.float32(2.0 ** -30)
    assert fma(a, b, 1.0 + 2.0 ** -24) == np.float32(1.0 + 2.0 ** -23)
    assert fma(np.float32(3.0), np.float32(5.0), np.float32(-15.0)) == 0.0


@pytest.mark.parametrize("far", [0, 10, 20, 24, 27, 28, 29, 30, 32, 36, 40])
def test_a_tile_is_taken_up_twice_at_most(far):
    x, unit = rows(far, 100)
    x[:, 1] *= np.float32(0.5)  # (a sum that is infinite by then stays as it is)
    for r in range(len(unit)):
        ref, total = np.float32(-np.inf), np.float32(0.0)
        for tile in range(2):
            ref, total, rounds = add_tokens(ref, total, x[r, tile], unit[r])
            assert rounds <= 2
        top = float(x[r].astype(np.float64).max() * np.float64(unit[r]))
        assert ref >= top - 8.0 - 2.0 ** -22 * abs(top) and ref <= top + 2.0 ** -22 * abs(top)


def test_without_that_limit_some_rows_never_end():
    x, unit = rows(29, 100)
    stuck = sum(add_tokens(np.float32(-np.inf), np.float32(0.0), x[r, 0], unit[r], most=1000)[2] == 59 for r in range(len(unit)))
    assert stuck > 5
    x, unit = rows(26, 100)
    assert all(add_tokens(np.float32(-np.inf), np.float32(0.0), x[r, 0], unit[r], most=1000)[2] < 4 for r in range(len(unit)))
