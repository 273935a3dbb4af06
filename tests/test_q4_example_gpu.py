"""The example that runs the 4-bit operators together."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [1, 5, 24])
def test_example(tokens):
    spec = importlib.util.spec_from_file_location("q4_block", os.path.join(ROOT, "examples", "q4_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    # h is kept to 16 bits of significand, sums are fp32
    assert mod.main(tokens) < 2.0 ** -15
