"""The gated feed-forward block from training to serving, as a user runs it
(examples/ffn_block.py), at small sizes."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ffn_block.py")


@pytest.mark.parametrize("G", [64, 128])
def test_train_pack_serve(G):
    spec = importlib.util.spec_from_file_location("ffn_block", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, error, apart = example.run(rows=150, model=256, hidden=640, G=G, steps=6)
    assert losses[-1] < losses[0]
    # Against bf16 weights: code * scale and h are rounded to bf16 (relative
    # 2^-9 on either side of each element), sums of hundreds of terms; an
    # element's error stays below a few times 2^-8 of the row's size.
    assert error < 2 ** -6
    # h of a row is rounded to bf16 after sums in another order: a half-ulp
    # apart (2^-8) where that falls on a boundary.
    assert apart < 2 ** -8
