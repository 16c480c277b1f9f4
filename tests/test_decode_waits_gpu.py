"""Bounded waits of the attention over latents: a wait that runs out (kvx_cache_inject_stall) ends in KVX_ETIMEDOUT, with the
CTA's copies and products waited for, and the next call on the same handle is right."""
import pytest

from test_decode_gpu import HND, NHD, Attend, kvx, torch

pytestmark = pytest.mark.gpu

PARTS = {"scores": 1, "sums": 2, "softmax": 3, "copies": 4}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


# shards 2: the kernel of warp products
@pytest.mark.parametrize("value,group,shards", [("bf16", 16, 1), ("f16", 32, 1), ("e4m3", 16, 1), ("e4m3", 32, 1), ("bf16", 16, 2),
                                                ("e4m3", 16, 2)])
@pytest.mark.parametrize("part", sorted(PARTS))
def test_a_wait_that_runs_out_is_reported(part, value, group, shards):
    case = Attend([19000, 0, 9000, 70], value=value, planes=1, shards=shards, hps=1, group=group, dim=576, v_dim=512, bs=64)
    out, lse = case.run()
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    kvx.kvx_cache_inject_stall(case.cache, PARTS[part])
    case.run()
    with pytest.raises(kvx.KvxError) as ei:
        kvx.kvx_cache_status(case.cache)
    assert ei.value.status == kvx.KVX_ETIMEDOUT
    again, lse2 = case.run()                                               # the hook fires once
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    kvx.kvx_cache_destroy(case.cache)


@pytest.mark.parametrize("layout", [NHD, HND])
def test_one_tile_and_a_wait_that_runs_out(layout):
    case = Attend([5], value="e4m3", planes=1, hps=1, group=16, dim=576, v_dim=512, bs=64, layout=layout)
    out, _ = case.run()
    for part in PARTS.values():
        kvx.kvx_cache_inject_stall(case.cache, part)
        case.run()
        with pytest.raises(kvx.KvxError):
            kvx.kvx_cache_status(case.cache)
    assert torch.equal(case.run()[0], out)
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
