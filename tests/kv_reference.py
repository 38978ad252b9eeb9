"""Attention over a quantized cache in 64 bits, with element-wise error bounds of the kernels' arithmetic.

Notation: o = sum_j p_j v_j over the tokens a row sees, v_j and k_j = low_j +
s_j c_j, size = sum_j p_j |v_j|.  An output is rounded to bf16, 8 significant
bits (2^-8 of it: 1 + 2^-8 becomes 1); what stands before that rounding is off by at most

few query rows (max_q * G <= 32):
    2^-11 sum_j p_j s_j |c_j - z|   each weight p_j s_j rounded to fp16 before it meets the centred code (z: 8, 128)
  + sum_j r_j (|v_j| + |o|) / (1 - sum_j r_j),  r_j = p_j (e^delta_j - 1)
                                    the logits, each off by delta_j at most: exact products, D / 16 fp32 accumulations
                                    and the scaling (or the same with every delta_j taken against the largest weight's,
                                    whose own r_j is then 0: logits so large that they are off by more than 1 in common),
                                    delta_j = 2^-18 scale (s_j sum_d |q_d| |c_jd - z| + |low_j + z s_j| sum_d |q_d|)
  + 2^-14 size                      exp2, fp32 sums over the tokens
  + 2^-32 n max_j |v_j|             weights that fp16 holds as subnormal numbers
many:
    (2^-11 + 2^-11) size + 2^-20 sum_j p_j max_d |v_jd|    P rounded to fp16, V rounded to fp16: 2^-11 of an element,
                                    and 2^-25 of 2^-5, which a token's largest element is brought to at least
  + the same of the logits          K rounded likewise, fp32 accumulation:
                                    delta_j = scale (1.01 * 2^-11 sum_d |q_d| |k_jd| + 2^-20 max_d |k_jd| sum_d |q_d|)
  + 2^-14 size
  + n (2^-32 max_j |v_j| + 2^-43 max over the whole sequence of |v|)   weights that fp16 holds as subnormal numbers,
                                    less 2^12 where a token's values are far below the largest around it
"""

from __future__ import annotations

import torch


def attended(q, codes, scale, low, n_q, window, softmax_scale, wide, centre):
    """(out, bound) fp64 [n_q, Hq, D] of one sequence: q [n_q, Hq, D]; codes [2, n, H, D], scale and low [2, n, H]."""
    q = torch.as_tensor(q, dtype=torch.float64)
    c = torch.from_numpy(codes.astype("float64"))
    s, lo = (torch.from_numpy(x.astype("float64")) for x in (scale, low))
    n, heads, d = c.shape[1:]
    g = q.shape[1] // heads
    out, bound = torch.zeros_like(q), torch.full_like(q, 1e-37)
    if n == 0 or n_q == 0:
        return out, bound
    kv = lo[..., None] + s[..., None] * c
    j, p = torch.arange(n), torch.arange(n - n_q, n)[:, None]
    see = j <= p
    if window:
        see &= j > p - window
    count = see.sum(-1)[:, None, None].double()
    for h in range(heads):
        k, v = kv[0, :, h], kv[1, :, h]
        qh = q[:, h * g:(h + 1) * g]
        aq = qh.abs()
        logits = softmax_scale * torch.einsum("igd,jd->igj", qh, k)
        w = torch.softmax(logits.masked_fill(~see[:, None], float("-inf")), -1)
        w = torch.where(see[:, None], w, torch.zeros(()).double())  # (rows that see nothing: 0, not a number otherwise)
        mix = lambda x: torch.einsum("igj,jd->igd", w, x)  # noqa: E731
        most = lambda x: torch.where(see[:, None], x, torch.zeros(()).double()).amax(-1)[..., None]  # noqa: E731
        o, size = mix(v), mix(v.abs())
        top = most(v.abs().amax(-1).expand(n_q, g, n))
        if wide:
            delta = 1.01 * 2.0 ** -11 * torch.einsum("igd,jd->igj", aq, k.abs())
            delta = delta + 2.0 ** -20 * aq.sum(-1)[..., None] * k.abs().amax(-1)
            err = 2.0 ** -10 * size + 2.0 ** -20 * mix(v.abs().amax(-1, keepdim=True).expand(n, d))
            err = err + count * (2.0 ** -32 * top + 2.0 ** -43 * v.abs().max())
        else:
            mid = (lo[0, :, h] + centre * s[0, :, h]).abs()
            delta = torch.einsum("igd,jd->igj", aq, s[0, :, h, None] * (c[0, :, h] - centre).abs())
            delta = 2.0 ** -18 * (delta + aq.sum(-1)[..., None] * mid)
            err = 2.0 ** -11 * mix(s[1, :, h, None] * (c[1, :, h] - centre).abs()) + count * 2.0 ** -32 * top
        log_p = torch.log_softmax(logits.masked_fill(~see[:, None], float("-inf")), -1)
        delta = abs(softmax_scale) * delta
        best = log_p.argmax(-1, keepdim=True)
        shifts = [delta, (delta + delta.gather(-1, best)).scatter(-1, best, 0.0)]  # (a common factor of the weights drops out)
        moved = []
        for shift in shifts:
            r = torch.where(see[:, None], torch.exp(log_p + shift) - w, torch.zeros(()).double())
            total = r.sum(-1)[..., None]
            e = (torch.einsum("igj,jd->igd", r, v.abs()) + total * o.abs()) / (1 - total)
            moved.append(torch.where((total < 1) & torch.isfinite(e), e, torch.full_like(e, float("inf"))))
        err = err + torch.minimum(*moved)
        err = err + 2.0 ** -14 * size
        out[:, h * g:(h + 1) * g] = o
        bound[:, h * g:(h + 1) * g] += 2.0 ** -8 * o.abs() + 1.01 * err
    return out, bound


def check(problem, y, window=0, scale=None, bar=None):
    """Holds the output y of a test_gpu_kv_cache.Problem to its bounds, and with `bar` to that relative Frobenius norm.
    Returns the share of elements whose bound says something (is below the largest value)."""
    scale = problem.d ** -0.5 if scale is None else scale
    y, at, err, ref, told = y.double().cpu(), 0, 0.0, 0.0, 0
    assert torch.isfinite(y).all()
    for (c, s, low), nq in zip(problem.seqs, problem.nqs):
        o, bound = attended(problem.q[at:at + nq].double(), c, s, low, nq, window, scale, problem.wide,
                            2 ** (problem.bits - 1))
        off = (y[at:at + nq] - o).abs()
        assert (off <= bound).all(), f"off by {(off / bound).max():.3g} of the bound"
        err += float((off ** 2).sum())
        ref += float((o ** 2).sum())
        if c.size:
            told += int((bound < float(abs(low[1]).max() + 256 * abs(s[1]).max())).sum())
        at += nq
    if bar is not None:
        assert err <= bar ** 2 * ref, f"relative error {(err / ref) ** 0.5:.2e}"
    return told / max(y.numel(), 1)
