"""Oracle of the quantized key/value cache, in numpy: quantization with the
contract's own fp32 operations (numpy's are IEEE, correctly rounded), and
everything behind it in 64 bits."""

from __future__ import annotations

import numpy as np

__all__ = ["quantize", "pack", "unpack", "values", "attention", "Attended"]


def quantize(x: np.ndarray, bits: int):
    """(codes uint8 [..., D], scale fp32 [...], low fp32 [...]) of fp32 rows."""
    x = np.asarray(x, np.float32)
    levels = np.float32(2 ** bits - 1)
    low = x.min(-1)
    r = (x.max(-1) - low) / levels
    # the smallest bf16 >= r: clear the low 16 bits, one step up where that lost something
    b = r.view(np.uint32)
    up = (b >> 16) + ((b & 0xFFFF) != 0)
    scale = (up << 16).astype(np.uint32).view(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((x - low[..., None]) / scale[..., None])
    c = np.where(scale[..., None] > 0, c, 0).clip(0, float(levels))
    return c.astype(np.uint8), scale, low


def pack(codes: np.ndarray, bits: int) -> np.ndarray:
    if bits == 8:
        return codes
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray, bits: int) -> np.ndarray:
    if bits == 8:
        return packed
    out = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def values(codes: np.ndarray, scale: np.ndarray, low: np.ndarray) -> np.ndarray:
    """fp64 values of unpacked codes."""
    return low[..., None].astype(np.float64) + scale[..., None].astype(np.float64) * codes


class Attended:
    """Result of attention() for one sequence, fp64 [n_q, Hq, D]: the output,
    and the magnitudes its error bounds are made of."""

    def __init__(self, n_q, hq, d):
        self.out = np.zeros((n_q, hq, d))
        self.weighted = np.zeros((n_q, hq, d))  # sum_j p_j |v_j - centre_j|: what rounding p_j s_j scales with
        self.size = np.zeros((n_q, hq, d))      # sum_j p_j |v_j|
        self.logit = np.zeros((n_q, hq))        # max_j softmax_scale sum_d |q_d| |k_jd|
        self.flush = np.zeros((n_q, hq, 1))     # visible tokens times the largest magnitude of their value rows
        self.mid = np.zeros((n_q, hq, 1))       # sum_j p_j |centre_j| of the values
        self.mid_logit = np.zeros((n_q, hq))    # max_j softmax_scale sum_d |q_d| |centre_j| of the keys
        self.biased = np.zeros((n_q, hq))       # max_j softmax_scale (sum_d |q_d| s_j (c + 128) + |low_j - 128 s_j| |sum q|)


def attention(q, codes, scale, low, n_q, window, softmax_scale, centre=8) -> Attended:
    """One sequence: q [n_q, Hq, D]; codes [2, n, H, D], scale and low [2, n, H]
    of its n cached tokens, the queries being the last n_q."""
    _, n, heads, d = codes.shape
    hq = q.shape[1]
    a = Attended(n_q, hq, d)
    kv = values(codes, scale, low)
    s64, l64 = scale.astype(np.float64), low.astype(np.float64)
    q = np.asarray(q, np.float64)
    for h in range(hq):
        c = h // (hq // heads)
        k, v = kv[0, :, c], kv[1, :, c]
        k_mid, v_mid = (np.abs(l64[x, :, c] + s64[x, :, c] * centre) for x in (0, 1))
        mid = np.abs(s64[1, :, c, None] * (codes[1, :, c].astype(np.float64) - centre))
        for i in range(n_q):
            p = n - n_q + i
            lo = max(0, p - window + 1) if window else 0
            if p < 0 or lo > p:
                continue
            see = slice(lo, p + 1)
            x = softmax_scale * (k[see] @ q[i, h])
            w = np.exp(x - x.max())
            w /= w.sum()
            a.out[i, h] = w @ v[see]
            a.weighted[i, h] = w @ mid[see]
            a.size[i, h] = w @ np.abs(v[see])
            a.mid[i, h] = w @ v_mid[see]
            a.flush[i, h] = len(w) * np.abs(v[see]).max()
            size = abs(softmax_scale)
            a.logit[i, h] = size * (np.abs(k[see]) @ np.abs(q[i, h])).max()
            a.mid_logit[i, h] = size * (k_mid[see] * np.abs(q[i, h]).sum()).max()
            bias = s64[0, see, c] * ((codes[0, see, c] + 128.0) @ np.abs(q[i, h])) + np.abs(
                l64[0, see, c] - 128 * s64[0, see, c]) * abs(q[i, h].sum())
            a.biased[i, h] = size * bias.max()
    return a
