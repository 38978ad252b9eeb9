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
