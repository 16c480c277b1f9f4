"""Tables as wide as max_blocks can be, of which rows hold their first pages: behind those nothing is read."""
import numpy as np
import pytest

import page_reference as ref
from test_pages_gpu import batch, dev, ints, kvx, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("width", [2 ** 31 - 1, 2 ** 31 - 127, 2 ** 31 - 128, 2 ** 31 - 129, 2 ** 30])
def test_free(width):
    bs = 16
    table, lens, n_blocks = batch(1, bs, 5000, 5, idle=0)
    assert lens[0] > 1000
    refs, free, result = ints(n_blocks), ints(n_blocks), ints(3, dtype=torch.int64)
    kvx.kvx_pages_free(dev(table), width, width, dev(lens), 1, bs, n_blocks, refs, free, result)
    want = ref.free(table, lens, bs, n_blocks)
    assert result.tolist() == want[2] and want[2][2] == kvx.KVX_OK
    assert np.array_equal(refs.cpu().numpy(), want[0]) and np.array_equal(free[:len(want[1])].cpu().numpy(), want[1])
