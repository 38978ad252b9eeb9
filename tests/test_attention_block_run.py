"""The budgets that the example's block refuses."""

from __future__ import annotations

import importlib.util
import os

import pytest

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
