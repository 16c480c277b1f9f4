"""Batches that kvx_cache_attend_shared gives to kvx_cache_attend: the groups are not looked at."""
import pytest

from shared_case import Shared
from test_decode_gpu import kvx, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("off,prefix", [([0, 3, 2, 5], None), ([-1, 2, 4, 5], None), ([0, 2 ** 31 - 1, 4, 5], None), ([0, 2, 4, 5], [300, -5, 50])])
def test_groups_are_read_where_the_batch_shares(off, prefix):
    case = Shared([(300, [0, 60]), (200, [1, 1]), 50], dim=64)
    case.shared()
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    for max_blocks, n_launches, status in ((case.width, 1, kvx.KVX_OK), (None, 3, kvx.KVX_ERANGE)):
        before = kvx.kvx_launch_count()
        got = case.shared(off=off, prefix=prefix, max_blocks=max_blocks)
        assert kvx.kvx_launch_count() - before == n_launches
        case.check_parts(*got)
        assert kvx.kvx_cache_status(case.cache) == status
