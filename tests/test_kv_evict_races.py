"""Eviction (``csrc/kv_evict.cu``: ``kv_select_kernel``) of weights that change
while they are read.  Contexts too long for shared memory are read from memory
in each pass: three for the threshold's digits, one that counts, one that gives
the kept tokens their slots.  A caller that lets them change meanwhile gets
tokens of its own choosing, but nothing may be written outside its row."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_linear_gb300 import capi

BITS = ((21, 2047), (10, 2047), (0, 1023))


def slots(keys, budget):
    """Slots of the kept tokens as the kernel gives them out, from the keys (uint32) that each of the five passes reads."""
    left, value, known = budget, 0, 0
    for k, (shift, digits) in zip(keys, BITS):
        hist = np.bincount((k[(k & known) == value] >> shift) & digits, minlength=digits + 1)
        above = 0
        for d in range(digits, -1, -1):
            if above < left <= above + hist[d]:
                value, left = value | d << shift, left - above
                break
            above += hist[d]
        known |= digits << shift
    k = keys[4]
    sure, tie = k > value, k == value
    s, t = np.cumsum(sure) - sure, np.cumsum(tie) - tie
    return (s + np.minimum(t, left))[sure | (tie & (t < left))]


def test_model_of_still_weights():
    rng = np.random.default_rng(0)
    for n, budget, most in ((1000, 300, 1 << 32), (500, 499, 7), (300, 1, 1 << 20)):
        k = rng.integers(0, most, n, dtype=np.uint32)
        assert slots([k] * 5, budget).tolist() == list(range(budget))


def test_model_of_changing_weights_leaves_the_row():
    """So the kernel holds a slot to the row."""
    rng = np.random.default_rng(1)
    k = rng.integers(0, 1 << 30, 1000, dtype=np.uint32)
    assert slots([k, k, k, k, k + np.uint32(1 << 30)], 300).max() >= 300


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_nothing_is_written_outside_the_row(cuda_device, in_place):
    """Another stream changes the weights all the while."""
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    n, page, heads, budget = 150001, 256, 2, 3000
    width = -(-n // page)
    codes, params = capi.kv_cache_alloc(width + 12, heads, page, 64)
    codes.zero_(), params.zero_()
    table = torch.arange(width, dtype=torch.int32, device="cuda")[None]
    spare = torch.arange(width, width + 12, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    weights = torch.rand((width + 12, heads, page), device="cuda")
    around = torch.full((n + heads * budget + n,), -77, dtype=torch.int32, device="cuda")
    kept = around[n:n + heads * budget].view(1, heads, budget)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(40):
        with torch.cuda.stream(other):
            for by in (3.0, -1.0, 0.25, 1e6, 1e-9):
                weights[: width].mul_(by)
        new, _ = capi.kv_cache_evict(codes, params, weights, table, lens, budget, first=4, last=64, kept=kept,
                                     new_table=None if in_place else spare)
        assert new.tolist() == [budget]
    torch.cuda.synchronize()
    assert (around[:n] == -77).all() and (around[n + heads * budget:] == -77).all()
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
