"""The example that trains a dense block, converts it and serves it, run in small."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
def test_train_convert_serve():
    import dense_to_mxfp4
    r = dense_to_mxfp4.main(tokens=192, hidden=256, d_ff=128, steps=40)
    assert r["last_loss"] < 0.6 * r["first_loss"]
    # a 4-bit value is off by at most a quarter of itself at its block's fine end, about a tenth in
    # the mean: one such operand a product, or three products of two
    assert r["mxfp4_down"] < 0.25 and r["mxfp4_block"] < 0.45 and r["mxfp4_experts"] < 0.45
