"""The example that runs the training losses together."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [1, 33, 256])
def test_example(tokens):
    spec = importlib.util.spec_from_file_location("expert_losses", os.path.join(ROOT, "examples", "expert_losses.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    loss, dX, dW, dR = mod.main(tokens)
    # the head's gradient is fp32; the router's logits' gradient is rounded to bf16 on its way: half a step, 2^-8
    assert loss < 1e-4 and dW < 1e-4 and dX < 2.0 ** -8 and dR < 2.0 ** -8
