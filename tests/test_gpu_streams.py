"""Memory that a call allocates belongs to the stream the call runs on: torch
gives a freed block out again in the order of its own stream only, so a block of
another stream may still be in use there."""

from __future__ import annotations

import pytest
import torch

from int8_quantized_linear_gb300 import capi
from tests.test_gpu_kv_cache import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    from int8_quantized_linear_gb300 import build
    build.build()
    capi.lib()
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    yield
    assert capi.i8ql_get_device_error() == capi.I8QL_OK


@pytest.fixture
def allocations(monkeypatch):
    """The raw handles of the streams that were current when torch.empty was called."""
    seen, empty = [], torch.empty

    def recording(*args, **kwargs):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kwargs)

    monkeypatch.setattr(torch, "empty", recording)
    return seen


def _streams():
    """(argument, raw handle): none given, a stream, its handle, the default stream by its handle."""
    side = torch.cuda.Stream()
    return [(None, torch.cuda.current_stream().cuda_stream), (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream),
            (0, 0)]


@pytest.mark.parametrize("which", range(4))
def test_attention_workspace(allocations, which):
    arg, handle = _streams()[which]
    p = Problem([300, 20000, 47], [1, 4, 2], 8, 2, 128, 4, 16, 77)
    q, out = p.q.cuda(), torch.zeros((7, 8, 128), dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(torch.cuda.Stream()):  # the default stream is not the current one either
        torch.cuda.synchronize()
        if which == 0:
            handle = torch.cuda.current_stream().cuda_stream
        allocations.clear()
        p.run(q=q, out=out, stream=arg)
        assert allocations == [handle]
        torch.cuda.synchronize()
    p.check(out)
