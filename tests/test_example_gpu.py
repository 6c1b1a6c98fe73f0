"""The example runs the operators together: the loss falls far below that of
random guessing, and tokens scored one at a time agree with the batch."""
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_bigram_lm(dtype):
    import bigram_lm
    losses, gap = bigram_lm.main(["--steps", "60", "--vocab", "1003", "--hidden", "256", "--dtype", dtype])
    assert abs(losses[0] - math.log(1003)) < 1.0
    # 60 batches of 2048 show every (token, successor) pair about 30 times
    assert losses[-1] < 0.5 * losses[0]
    # the single-row and the batch kernels sum in different orders: a few roundings of x apart
    assert gap < 0.05
