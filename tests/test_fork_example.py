"""The example of several answers to one prompt runs, and its checks of itself hold: forked and compacted pages, rotated
appends and attention over a shared prefix, together, in a captured step."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# Outputs are means of values, N(0, 1) up to about 5: half a unit of bf16 there is 2^-6. A rotated value is within half a unit of its
# size, 2^-8, and of 32-bit arithmetic on numbers up to about 10 (10 * 2^-19 of at least 1e-2): 2^-8 + 2^-9 in all.
@pytest.mark.parametrize("prompt,answers", [(500, 12), (512, 7)])
def test_small_batches_read_the_prompt_themselves(prompt, answers):
    """Two megabytes of pages: below what sharing is worth."""
    import fork_shared_prompt
    out, turned = fork_shared_prompt.main(steps=30, prompt=prompt, answers=answers)
    assert out < 2.0 ** -6 and turned < 2.0 ** -8 + 2.0 ** -9


def test_shared_prompt():
    """240 MB that would be read again."""
    import fork_shared_prompt
    before = fork_shared_prompt.kvx.kvx_launch_count()
    out, turned = fork_shared_prompt.main(steps=8, prompt=5005, answers=48)
    assert out < 2.0 ** -6 and turned < 2.0 ** -8 + 2.0 ** -9
    # 12 around the steps; the first step and the capture: free, slots, and of each of two layers a rotated append and three of the attention
    assert fork_shared_prompt.kvx.kvx_launch_count() - before == 12 + 2 * (2 + 2 * 4)
