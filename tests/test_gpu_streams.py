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


def _calls():
    """name -> (call of the binding that makes all its outputs itself, how many it makes)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    bf = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, w = bf(16, 256), bf(256, 256)
    qx, sx = capi.quantize_act_per_token_int8(x)
    qw, sw = capi.quantize_weight_per_channel_int8(w)
    fx, fsx = capi.quantize_act_per_token_fp8(x)
    fw, fsw = capi.quantize_weight_per_channel_fp8(w)
    w4, s4 = capi.quantize_weight_w4_g128(w)
    logits = torch.randn((16, 8), generator=g, device="cuda")
    offsets, row_token, token_row, slot_weight = capi.moe_route_topk(logits, 2, 1)
    gu, sgu = (t.view(9, 256, -1) for t in capi.quantize_weight_per_channel_int8(bf(9 * 256, 256)))
    dn, sdn = (t.view(9, 256, -1) for t in capi.quantize_weight_per_channel_int8(bf(9 * 256, 128)))
    sgu, sdn = sgu.view(9, 256), sdn.view(9, 256)
    rows = bf(48, 256)
    codes, params = capi.kv_cache_alloc(4, 2, 16, 64)
    k, slots = bf(50, 2, 64), torch.arange(50, device="cuda")
    capi.kv_cache_store(k, k, slots, codes, params)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([50], dtype=torch.int32, device="cuda")
    q = bf(1, 4, 64)
    return {
        "quantize_act_per_token_int8": (lambda s: capi.quantize_act_per_token_int8(x, stream=s), 2),
        "quantize_weight_per_channel_int8": (lambda s: capi.quantize_weight_per_channel_int8(w, stream=s), 2),
        "w8a8_linear": (lambda s: capi.w8a8_linear(x, qw, sw, stream=s), 1),
        "w8a8_gemm": (lambda s: capi.w8a8_gemm(qx, sx, qw, sw, stream=s), 1),
        "w8a16_gemm": (lambda s: capi.w8a16_gemm(x, qw, sw, stream=s), 1),
        "grouped_w8a16_gemm": (lambda s: capi.grouped_w8a16_gemm(rows, offsets, gu, sgu, stream=s), 1),
        "quantize_act_per_token_fp8": (lambda s: capi.quantize_act_per_token_fp8(x, stream=s), 2),
        "quantize_weight_per_channel_fp8": (lambda s: capi.quantize_weight_per_channel_fp8(w, stream=s), 2),
        "w8a8_fp8_gemm": (lambda s: capi.w8a8_fp8_gemm(fx, fsx, fw, fsw, stream=s), 1),
        "w8a8_fp8_linear": (lambda s: capi.w8a8_fp8_linear(x, fw, fsw, stream=s), 1),
        "quantize_weight_w4_g128": (lambda s: capi.quantize_weight_w4_g128(w, stream=s), 2),
        "w4a16_gemm": (lambda s: capi.w4a16_gemm(x, w4, s4, stream=s), 1),
        "moe_route_topk": (lambda s: capi.moe_route_topk(logits, 2, 1, stream=s), 4),
        "grouped_w8a16_silu_mul": (lambda s: capi.grouped_w8a16_silu_mul(x, row_token, offsets, gu, sgu, stream=s), 1),
        "moe_combine": (lambda s: capi.moe_combine(rows, token_row, slot_weight, stream=s), 1),
        "moe_expert_mlp_w8a16": (lambda s: capi.moe_expert_mlp_w8a16(x, logits, 2, 1, gu, sgu, dn, sdn, stream=s), 1),
        "kv_cache_load": (lambda s: capi.kv_cache_load(codes, params, slots, 64, stream=s), 2),
        "kv_cache_attention": (lambda s: capi.kv_cache_attention(q, codes, params, table, lens, stream=s), 1),
    }


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("name", ["quantize_act_per_token_int8", "quantize_weight_per_channel_int8", "w8a8_linear", "w8a8_gemm",
                                  "w8a16_gemm", "grouped_w8a16_gemm", "quantize_act_per_token_fp8",
                                  "quantize_weight_per_channel_fp8", "w8a8_fp8_gemm", "w8a8_fp8_linear",
                                  "quantize_weight_w4_g128", "w4a16_gemm", "moe_route_topk", "grouped_w8a16_silu_mul",
                                  "moe_combine", "moe_expert_mlp_w8a16", "kv_cache_load", "kv_cache_attention"])
def test_outputs(allocations, name, which):
    arg, handle = _streams()[which]
    call, outputs = _calls()[name]
    want = call(None)
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.synchronize()
        if which == 0:
            handle = torch.cuda.current_stream().cuda_stream
        allocations.clear()
        got = call(arg)
        assert allocations == [handle] * outputs
        torch.cuda.synchronize()
    for a, b in zip(*((t,) if torch.is_tensor(t) else t for t in (got, want))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("handle", [False, True])
def test_a_block_just_freed_is_not_written_by_another_stream(handle):
    p = Problem([300, 20000, 47], [1, 4, 2], 8, 2, 128, 4, 16, 77)
    q, slots = p.q.cuda(), torch.arange(333, device="cuda")
    st = torch.cuda.Stream()
    arg = st.cuda_stream if handle else st
    torch.cuda.synchronize()

    def freed(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").data_ptr()

    at = freed(7, 8, 128)
    y = p.run(q=q, stream=arg)
    assert y.data_ptr() != at
    at = freed(333, 2, 128)
    k, v = capi.kv_cache_load(p.codes, p.params, slots, 128, stream=arg)
    assert at not in (k.data_ptr(), v.data_ptr())
    torch.cuda.synchronize()
    p.check(y)
