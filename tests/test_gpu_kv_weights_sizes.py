"""GPU tests of what kv_cache_weights takes of workspace: a call takes what the
query of the same sizes says, also where the bound on a sequence's query tokens
exceeds those there are."""

from __future__ import annotations

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


@pytest.mark.parametrize("nqs,hq,heads,tokens,max_q", [
    ([1, 1], 32, 8, 1 << 17, 16),       # two kernels for few rows, one launch's rows by the bound
    ([1, 1], 32, 8, 1 << 17, 64),       # the bound is a prompt's
    ([256], 8, 8, 1 << 20, 1024),
    ([100, 33], 4, 1, 1 << 16, 5000),
    ([1, 1, 1], 4, 4, 4096, 8),
])
def test_workspace_of_a_bound_above_the_queries(nqs, hq, heads, tokens, max_q):
    page, d = 256, 64
    c = Cache([300 + n for n in nqs], hq, heads, d, 4, page, nqs, wide=tokens // page - 2)
    assert c.table.shape[1] * page >= tokens - 512
    sizes = (len(nqs), sum(nqs), hq, heads, d, 4, page, c.table.shape[1])
    told = capi.i8ql_kv_weights_workspace(*sizes, max_q)
    assert told == capi.i8ql_kv_weights_workspace(*sizes, sum(nqs))
    space = torch.empty(max(told, 1), dtype=torch.uint8, device="cuda")
    c.check(c.weigh(max_q=max_q, workspace=space))
    if told:
        with pytest.raises(capi.I8qlError):
            c.weigh(max_q=max_q, workspace=space[: told - 1])
