"""The example of a decode worker runs: push, then graph-captured steps of slot map, append and attention over block
borders, every output within bf16's rounding of the 64-bit check that the example makes itself."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_decode_after_push():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import decode_after_push
    # outputs of one cached token are its values, N(0, 1) up to about 5: half a unit of bf16 there is 2^-6, and a weight's
    # rounding is far below it
    assert decode_after_push.main(steps=70) < 2.0 ** -6
