"""The example block end to end: it learns, and its tokens do not depend on
each other (bit for bit where the grouped GEMM takes the same path)."""

import importlib.util
import os

import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


def test_block_trains_and_decodes():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    losses, whole, single = block.main(tokens=256, width=256, hidden=128, experts=8, k=2, steps=6,
                                       say=lambda text, flush: say(text))
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    # one bf16 rounding of y and of the rows before it apart at most
    assert float((whole - single).abs().max()) <= 2 ** -7 * float(whole.abs().max())
