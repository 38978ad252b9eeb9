"""GPU tests of attention weights summed per token (kv_cache_weights) whose
logits are large: up to where their fp32 spacing passes the softmax's own units
and beyond."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import capi
from tests.test_gpu_kv_evict import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    from int8_quantized_linear_gb300 import build
    build.build()
    capi.lib()
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    yield
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


def rescale(c, i, far):
    """The keys of sequence i of a Cache times 2^far (exactly)."""
    codes, s, low = c.seqs[i]
    c.seqs[i] = (codes, s * np.float32(2.0 ** far), low * np.float32(2.0 ** far))
    j = np.arange(c.lens[i])
    pages, off = torch.from_numpy(c.table[i, j // c.page]).long().cuda(), torch.from_numpy(j % c.page).cuda()
    c.params[pages, 0, :, off] *= 2.0 ** far


def of(c, w, i):
    """Weights [heads, tokens] of sequence i."""
    j = np.arange(c.lens[i])
    return w.cpu().double().numpy()[c.table[i, j // c.page], :, j % c.page].T


@pytest.mark.parametrize("bits,d", [(4, 128), (8, 128), (4, 64), (8, 64)])
@pytest.mark.parametrize("far", [24, 29, 33, 40])
def test_many_rows_end(bits, d, far):
    """Logits of any size: the call ends, and the other sequences of the call are as they are without them."""
    c = Cache([900, 300], 4, 2, d, bits, 32, [150, 60], seed=far)
    want = of(c, c.weigh(), 1)
    rescale(c, 0, far)
    assert np.array_equal(of(c, c.weigh(), 1), want)


# Forms of few query rows: one launch of 8, 16 and 32 rows, one and several CTAs a cluster; two kernels of 8, 16, 32
# and twice 32 rows.  (lens, queries, query heads, heads, page, pages more in the table)
FEW = [
    ([1100, 40], [1, 1], 8, 2, 32, 0),
    ([5000, 130], [1, 1], 4, 1, 64, 0),
    ([700, 90], [4, 3], 8, 2, 16, 0),
    ([500, 77], [7, 5], 8, 2, 32, 0),
    ([900, 300], [2, 1], 4, 1, 16, 5000),
    ([900, 300], [4, 1], 4, 1, 256, 300),
    ([600, 131], [8, 6], 8, 2, 16, 5000),
    ([800, 300], [15, 9], 8, 2, 64, 0),
]
SIZES = [0, 7, 16, 24, 28, 31, 33, 40, 70, 110]


def check_rows(c, w, each):
    """Weights are finite and not negative, and those of each sequence and head sum to its rows (all see some token).
    each: how far a row's may be off 1."""
    for i, nq in enumerate(c.nqs):
        x = of(c, w, i)
        assert np.isfinite(x).all() and (x >= 0).all()
        rows = nq * c.q.shape[1] // c.heads
        total = x.sum(1)
        # (a token's sum is rounded once for each row at most, a row's for each of its tokens and lanes)
        assert (np.abs(total - rows) <= rows * (each + (c.lens[i] + rows) * 2.0 ** -24)).all(), total / rows - 1


def check_pinned(c, w, scale):
    """Rows whose largest logit lies above the others by far more than logits may be off (2^-18 of the magnitudes that
    they add up): their weight is all that token's.  Returns their share of sequence 0's rows."""
    shares = []
    for i, nq in enumerate(c.nqs):
        pinned = rows = 0
        first = sum(c.nqs[:i])
        codes, s, low = (x.astype(np.float64) for x in c.seqs[i])
        q = c.q[first:first + nq].double().numpy()
        n, group = c.lens[i], q.shape[1] // c.heads
        k, size = low[..., None] + s[..., None] * codes, np.abs(low) + np.abs(s) * 2.0 ** c.bits
        least = np.zeros((c.heads, n))
        for t in range(nq):
            see = n - nq + t + 1
            for h in range(q.shape[1]):
                x = k[:see, h // group] @ q[t, h] * scale
                off = 2.0 ** -18 * scale * size[:see, h // group] * np.abs(q[t, h]).sum()
                best = int(x.argmax())
                apart = x[best] - off[best] - np.delete(x + off, best)
                rows += 1
                if see > 1 and apart.min() > 40:
                    pinned += 1
                    least[h // group, best] += 1.0
        assert (of(c, w, i) >= least * (1 - 2.0 ** -10)).all()
        shares.append(pinned / rows)
    return shares[0]


@pytest.mark.parametrize("bits,d", [(4, 128), (8, 64)])
@pytest.mark.parametrize("far", SIZES)
@pytest.mark.parametrize("form", range(len(FEW)))
def test_few_rows(form, far, bits, d):
    lens, nqs, hq, heads, page, wide = FEW[form]
    c = Cache(lens, hq, heads, d, bits, page, nqs, seed=form, wide=wide)
    rescale(c, 0, far)
    w = c.weigh()
    # exponentials are off by 2^-21, and exponents by their own rounding; references below 2^12 by 2^-25 of them, in each
    # kernel; larger ones not at all, as exponents are differences of the very products to the largest
    check_rows(c, w, 2.0 ** -19 + 2.0 ** -24 * min(2.0 ** (far + 5), 2.0 ** 12))
    assert far < 20 or check_pinned(c, w, d ** -0.5) > 0.5


def equal_keys(c, i):
    """All keys of sequence i as its first."""
    j = np.arange(c.lens[i])
    pages, off = torch.from_numpy(c.table[i, j // c.page]).long().cuda(), torch.from_numpy(j % c.page).cuda()
    c.codes[pages, 0, :, off] = c.codes[pages[0], 0, :, off[0]]
    c.params[pages, 0, :, off] = c.params[pages[0], 0, :, off[0]]


def uniform(c, i):
    """Weights of sequence i whose keys are all equal."""
    n, nq = c.lens[i], c.nqs[i]
    want = np.zeros(n)
    for t in range(nq):
        want[: n - nq + t + 1] += c.q.shape[1] // c.heads / (n - nq + t + 1)
    return want


@pytest.mark.parametrize("bits,d", [(4, 128), (8, 64)])
@pytest.mark.parametrize("far", SIZES)
@pytest.mark.parametrize("form", range(len(FEW)))
def test_few_rows_of_equal_keys(form, far, bits, d):
    """Equal logits, however large, share a row equally."""
    lens, nqs, hq, heads, page, wide = FEW[form]
    c = Cache(lens, hq, heads, d, bits, page, nqs, seed=form, wide=wide)
    rescale(c, 0, far)
    equal_keys(c, 0)
    w, want = of(c, c.weigh(), 0), uniform(c, 0)
    # (equal exponents, the same in both passes; rounded sums over the tokens and over the rows, a quotient)
    assert (np.abs(w / want - 1) <= (4 + lens[0] + nqs[0] * hq // heads) * 2.0 ** -24).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e4, 3e30])
@pytest.mark.parametrize("form", [0, 2, 4, 7])
def test_few_rows_of_any_scale(form, scale):
    lens, nqs, hq, heads, page, wide = FEW[form]
    for far in (0, 60, 100):
        if scale * 2.0 ** far > 2.0 ** 115:  # (logits past fp32 are nobody's)
            continue
        c = Cache(lens, hq, heads, 64, 4, page, nqs, seed=form, wide=wide)
        rescale(c, 0, far)
        check_rows(c, c.weigh(scale=scale), 2.0 ** -19 + 2.0 ** -12)


# Many query rows: both halves of a row block and one, several row blocks, several parts of the tokens, and a table so wide
# that row blocks share their sums.  (lens, queries, query heads, heads, page, pages more in the table, window)
MANY = [
    ([900, 300], [150, 60], 4, 2, 32, 0, 0),
    ([700, 131], [90, 131], 8, 2, 16, 0, 0),
    ([1500], [600], 3, 1, 64, 0, 0),
    ([1330, 40], [1030, 33], 4, 1, 256, 4096, 0),
    ([6000, 300], [17, 20], 16, 4, 64, 0, 0),
    ([1500, 300], [200, 70], 4, 2, 32, 0, 100),
]


def near(far):
    """How far logits up to 2^12 may be off in a row's exponents, relative to each other: products rounded to 2^-24 of
    them where some row does not see some token, reference and logarithm of the sum rounded as one number."""
    return 2.0 ** -23 * min(2.0 ** (far + 5), 2.0 ** 13)


@pytest.mark.parametrize("bits,d", [(4, 128), (8, 128), (4, 64), (8, 64)])
@pytest.mark.parametrize("far", SIZES)
@pytest.mark.parametrize("form", range(len(MANY)))
def test_many_rows(form, far, bits, d):
    lens, nqs, hq, heads, page, wide, window = MANY[form]
    c = Cache(lens, hq, heads, d, bits, page, nqs, seed=form, wide=wide)
    rescale(c, 0, far)
    w = c.weigh(window)
    if window:
        seen = [np.arange(n) >= n - nq + 1 - window for n, nq in zip(lens, nqs)]
        for i in range(len(lens)):
            assert (of(c, w, i)[:, ~seen[i]] == -5.0).all()
        w = torch.where(w == -5.0, torch.zeros(()).cuda(), w)
    # (and logarithms and exponentials to 2^-19)
    check_rows(c, w, 2.0 ** -18 + near(far))
    assert far < 20 or window or check_pinned(c, w, d ** -0.5) > 0.5


@pytest.mark.parametrize("bits,d", [(4, 128), (8, 64)])
@pytest.mark.parametrize("far", SIZES)
@pytest.mark.parametrize("form", [0, 1, 2, 3, 4])
def test_many_rows_of_equal_keys(form, far, bits, d):
    lens, nqs, hq, heads, page, wide, _ = MANY[form]
    c = Cache(lens, hq, heads, d, bits, page, nqs, seed=form, wide=wide)
    rescale(c, 0, far)
    equal_keys(c, 0)
    w, want = of(c, c.weigh(), 0), uniform(c, 0)
    assert (np.abs(w / want - 1) <= 2.0 ** -18 + near(far) + (4 + lens[0] + nqs[0] * hq // heads) * 2.0 ** -24).all()


@pytest.mark.parametrize("scale", [-0.1, 1e-30, 1e-3, 1e4, 3e30])
@pytest.mark.parametrize("form", [0, 2, 4])
def test_many_rows_of_any_scale(form, scale):
    lens, nqs, hq, heads, page, wide, _ = MANY[form]
    for far in (0, 60, 100):
        if abs(scale) * 2.0 ** far > 2.0 ** 115:  # (logits past fp32 are nobody's)
            continue
        c = Cache(lens, hq, heads, 64, 4, page, nqs, seed=form, wide=wide)
        rescale(c, 0, far)
        check_rows(c, c.weigh(scale=scale), 2.0 ** -18 + near(12))


@pytest.mark.parametrize("bits,d", [(4, 128), (8, 64)])
def test_many_rows_near_and_far_together(bits, d):
    """Rows whose logits lie on both sides of where references are kept in another way, in one warp and one group, and
    rows that cross it from one tile to the next."""
    c = Cache([1390, 300], 4, 2, d, bits, 32, [150, 60], seed=1)
    by = 2.0 ** torch.arange(0, 15)[torch.arange(210) % 15]
    c.q = (c.q.float() * by[:, None, None]).to(torch.bfloat16)
    check_rows(c, c.weigh(), 2.0 ** -18 + near(12))
    rising = 2.0 ** np.repeat(np.arange(11), 128)  # a tile's keys twice the last one's
    for i, n in enumerate(c.lens):
        codes, s, low = c.seqs[i]
        j = np.arange(n)
        pages, off = torch.from_numpy(c.table[i, j // 32]).long().cuda(), torch.from_numpy(j % 32).cuda()
        c.params[pages, 0, :, off] *= torch.from_numpy(rising[:n]).to(torch.bfloat16).cuda()[:, None, None]
        c.seqs[i] = (codes, s * rising[:n, None].astype(np.float32), low * rising[:n, None].astype(np.float32))
    w = c.weigh()
    check_rows(c, w, 2.0 ** -18 + near(12))
