"""The example's block with a budget over more tokens than a sequence holds at a
time, and the budgets that it refuses."""

from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from int8_quantized_linear_gb300 import capi

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("budget,recent", [(10, 16), (15, 16), (8, -1)])
def test_recent_tokens_are_part_of_the_budget(example, budget, recent):
    with pytest.raises(ValueError, match="budget"):
        example.AttentionBlock(64, 1, 1, 64, budget=budget, recent=recent, device="cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("budget,recent", [(40, 16), (16, 16), (5, 2), (1, 0)])
def test_more_tokens_than_are_held(example, cuda_device, budget, recent):
    """Positions go on where lengths are cut: queries are turned by them, exactly, however many there are."""
    assert capi.i8ql_get_device_error() == capi.I8QL_OK
    freqs = capi.rotary_frequencies(64, 1e4)
    block = example.AttentionBlock(128, 4, 2, 64, pages=24, page_size=16, max_tokens=96, rotary=freqs, budget=budget,
                                   recent=recent)
    at = {"a": 0, "b": 0}
    for step, batch in enumerate([[("a", 50), ("b", 20)]] + [[("a", 30), ("b", 1)]] * 6 + [[("b", 1), ("a", 1)]] * 3):
        tokens = sum(n for _, n in batch)
        x = torch.randn((tokens, 128), generator=torch.Generator(device="cuda").manual_seed(step), device="cuda").bfloat16()
        y, _ = block.forward(x, batch)
        places = []
        for name, n in batch:
            places += range(at[name], at[name] + n)
            at[name] += n
        rows = capi.w8a16_gemm(x, *block.qkv).view(tokens, 8, 64)
        want = capi.rotary_apply(rows[:, :4], capi.rotary_table(freqs, torch.tensor(places, device="cuda")))
        assert torch.equal(block.last_q, want) and torch.isfinite(y.float()).all()
        block.cut([name for name, _ in batch])
        assert capi.i8ql_get_device_error() == capi.I8QL_OK
    assert at["a"] > 96 and all(n <= budget for n in block.lengths.values())
    assert len(block.free) + sum(map(len, block.pages.values())) == 24
