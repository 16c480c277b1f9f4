"""Queries and scales so small that their product is no 32-bit number: all positions weigh the same."""
import pytest

from shared_case import Shared
from test_decode_gpu import Attend, kvx, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


# Lengths that end inside a tile: a position behind the end must not count, whatever the scale.
@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("scale,power", [(-40, -80), (-60, -100), (-110, -100), (-120, -110), (-120, 0)])
def test_attend(value, scale, power):
    case = Attend([5, 131, 0, 700], value=value, dim=64, group=3, scale=2.0 ** scale)
    case.q = (case.q.double() * 2.0 ** (power if value != "f16" else max(power, -10))).to(case.iodtype)
    case.check(*case.run())
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("scale,power", [(-40, -80), (-60, -100), (-110, -100), (-120, -110), (-120, 0)])
def test_attend_shared(value, scale, power):
    case = Shared([(300, [1, 77]), (129, [0] * 40)], value=value, dim=128, group=4, scale=2.0 ** scale)
    case.q = (case.q.double() * 2.0 ** (power if value != "f16" else max(power, -10))).to(case.iodtype)
    case.check_parts(*case.shared())
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
