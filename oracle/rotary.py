"""Oracle of rotary positions, in numpy: angles in extended precision, and rows
turned with the contract's own fp32 operations (numpy's are IEEE, correctly
rounded)."""

from __future__ import annotations

import math

import numpy as np

__all__ = ["table", "turn", "turn64"]

_TWO_PI = (2 * math.pi, 2.4492935982947064e-16)  # 2 pi as the sum of two doubles


def table(freqs, positions, amplitude=1.0):
    """fp64 [P, 2F]: amplitude cos(p f), then amplitude sin(p f), of the exact product p f."""
    from fractions import Fraction
    turn = Fraction(_TWO_PI[0]) + Fraction(_TWO_PI[1])
    out = np.zeros((len(positions), 2 * len(freqs)))
    for i, f in enumerate(freqs):
        x = Fraction(float(f))
        for r, p in enumerate(positions):
            a = x * int(p)
            a -= turn * round(a / turn)
            out[r, i], out[r, len(freqs) + i] = math.cos(a), math.sin(a)
    return amplitude * out


def _pairs(x, rot, interleaved):
    t = x[..., :rot]
    return (t[..., 0::2], t[..., 1::2]) if interleaved else (t[..., : rot // 2], t[..., rot // 2:])


def _join(x, a, b, rot, interleaved):
    out = x.copy()
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2] = a, b
    else:
        out[..., : rot // 2], out[..., rot // 2: rot] = a, b
    return out


def turn(x, rows, interleaved, backward=False):
    """fp32 [T, heads, D] (bf16 values) turned by table rows [T, rot], before the last rounding to bf16."""
    x, rows = np.asarray(x, np.float32), np.asarray(rows, np.float32)
    rot = rows.shape[1]
    c, s = rows[:, None, : rot // 2], rows[:, None, rot // 2:]
    if backward:
        s = -s
    a, b = _pairs(x, rot, interleaved)
    return _join(x, a * c - b * s, b * c + a * s, rot, interleaved)


def turn64(x, rows, interleaved, backward=False):
    """The same in 64 bits throughout."""
    x, rows = np.asarray(x, np.float64), np.asarray(rows, np.float64)
    rot = rows.shape[1]
    c, s = rows[:, None, : rot // 2], rows[:, None, rot // 2:] * (-1 if backward else 1)
    a, b = _pairs(x, rot, interleaved)
    return _join(x, a * c - b * s, b * c + a * s, rot, interleaved)
