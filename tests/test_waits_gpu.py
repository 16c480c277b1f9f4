"""How late a wait ends that runs out: by the hooks of the attention kernels, whose limit is 1 ms."""
import pytest

from shared_case import Shared
from test_decode_gpu import Attend, kvx, torch

pytestmark = pytest.mark.gpu

# The limit, a quarter of a millisecond until the clock is read again, and as much for what is waited for after it: copies
# and products under way, whose waits have begun by then. The rest is for launches and for the call without a stall (0.1 ms).
LATEST_MS = 2.5


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def attend(case, out, lse):
    n, hq = len(case.lens), case.heads * case.group
    kvx.kvx_cache_attend(case.cache, 0, case.d_q, case.d_q.shape[1], case.d_table, case.d_table.shape[1], case.d_table.shape[1], case.d_len, n,
                         out, hq * case.v_dim, lse)


def attend_shared(case, out, lse):
    n, hq = len(case.lens), case.heads * case.group
    kvx.kvx_cache_attend_shared(case.cache, 0, case.d_q, hq * case.dim, case.d_table, case.d_table.shape[1], case.d_table.shape[1],
                                case.d_len, n, case.d_off, case.d_prefix, len(case.prefix), out, hq * case.dim, lse, case.space, case.space.numel())


def check(case, call, inject):
    out = torch.zeros((len(case.lens), case.heads * case.group * case.v_dim), dtype=case.iodtype, device="cuda")
    lse = torch.zeros((len(case.lens), case.heads * case.group), device="cuda")
    call(case, out, lse)
    want = out.clone()
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    inject()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    begin.record()
    call(case, out, lse)
    end.record()
    torch.cuda.synchronize()
    with pytest.raises(kvx.KvxError) as ei:
        kvx.kvx_cache_status(case.cache)
    assert ei.value.status == kvx.KVX_ETIMEDOUT
    assert 1.0 <= begin.elapsed_time(end) < LATEST_MS
    call(case, out, lse)
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK and torch.equal(out, want)


@pytest.mark.parametrize("value,shards", [("e4m3", 1), ("bf16", 1), ("e4m3", 2), ("bf16", 2)])
@pytest.mark.parametrize("part", [1, 2, 3, 4])
def test_latents(value, shards, part):
    case = Attend([19000, 0, 9000, 70], value=value, planes=1, shards=shards, hps=1, group=16, dim=576, v_dim=512, bs=64)
    case.run()
    check(case, attend, lambda: kvx.kvx_cache_inject_stall(case.cache, part))


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
@pytest.mark.parametrize("part", [1, 2, 3])
def test_shared_prefixes(value, part):
    case = Shared([(3000, [9] * 3), 50, (200, [1, 1])], value=value, dim=128, group=8, hps=1)
    case.shared()
    check(case, attend_shared, lambda: kvx.kvx_cache_inject_shared_stall(case.cache, part))
