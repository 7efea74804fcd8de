"""The behaviour-attention example: it trains, and its single-event answers
are the forward's rows."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_behaviour_attention_example():
    spec = importlib.util.spec_from_file_location("behaviour_attention",
                                                  os.path.join(ROOT, "examples", "behaviour_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, off = mod.main(users=60, steps=20)
    assert losses[-1] < losses[0]
    # outputs of magnitude below 4, rounded to bf16 twice (spacing 2^-6 there),
    # the same sums in another order
    assert off <= 2**-5
