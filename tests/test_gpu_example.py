"""The example block: it trains, and serves what it trained."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "hybrid_block.py")
    spec = importlib.util.spec_from_file_location("hybrid_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_hybrid_block():
    # the serving path rounds to bf16 where the training path does, in sums of
    # another order: a few spacings of 2^-8 of single values at most
    losses, error = example().main(train_steps=30, new_tokens=20, log=lambda s: None)
    assert losses[-1] < 0.9 * losses[0]
    assert error <= 2.0 ** -7
