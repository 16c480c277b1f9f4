"""Refusals of kvx_cache_attend_shared, none of which needs a GPU, and its workspace."""
import pytest

from test_decode_host import GEOM, LATENT, pool, refused

kvx = pytest.importorskip("disaggregated_prefill_decode_gb300.kvx")
A = 1 << 20                                                              # an address that is never read
CALL = dict(layer=0, q=A, q_stride=256, block_table=A, table_stride=8, max_blocks=8, seq_len=A, n_reqs=3, group_off=A, prefix_len=A,
            n_groups=1, out=A, out_stride=256, lse=A, workspace=A, workspace_bytes=1 << 40)


@pytest.mark.parametrize("bad", [
    dict(layer=2), dict(layer=-1), dict(n_reqs=-1), dict(n_reqs=(1 << 24) + 1), dict(max_blocks=-1), dict(table_stride=7), dict(q=None),
    dict(out=None), dict(seq_len=None), dict(block_table=None), dict(q_stride=248), dict(out_stride=248), dict(q_stride=1 << 41),
    dict(q=A + 8), dict(out=A + 8), dict(q_stride=260), dict(lse=A + 2), dict(seq_len=A + 1), dict(n_groups=-1),
    dict(n_groups=(1 << 24) + 1), dict(group_off=None), dict(prefix_len=None), dict(group_off=A + 2), dict(prefix_len=A + 1),
    dict(workspace=A + 8), dict(workspace_bytes=-1)])
def test_refusals(bad):
    c = kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16, n_q_heads=4)
    refused(kvx.kvx_cache_attend_shared, kvx.KVX_EINVAL, c, **{**CALL, **bad})


def test_no_requests_and_destroyed():
    c = kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16, n_q_heads=4)
    kvx.kvx_cache_attend_shared(c, **{**CALL, "n_reqs": 0, "workspace": None, "workspace_bytes": 0})
    for bad in ((-1, 1), (1, -1), ((1 << 24) + 1, 1), (1, (1 << 24) + 1)):
        refused(kvx.kvx_cache_shared_bytes, kvx.KVX_EINVAL, c, *bad)
    assert kvx._lib.kvx_cache_shared_bytes(c.handle, 2, 1, None) == kvx.KVX_EINVAL
    assert kvx.kvx_cache_shared_bytes(c, 1, 1) == 0 and kvx.kvx_cache_shared_bytes(c, 5, 0) == 0
    latent = kvx.kvx_cache_create(pool(LATENT), value_type=kvx.KVX_E4M3, v_dim=512)
    assert kvx.kvx_cache_shared_bytes(latent, 8, 2) == 0                   # latents do not share
    refused(kvx.kvx_cache_inject_shared_stall, kvx.KVX_EUNSUPPORTED, latent, 1)
    for part in (0, 4):
        refused(kvx.kvx_cache_inject_shared_stall, kvx.KVX_EINVAL, c, part)
    kvx.kvx_cache_destroy(c)
    refused(kvx.kvx_cache_attend_shared, kvx.KVX_EINVAL, c, **CALL)
    refused(kvx.kvx_cache_shared_bytes, kvx.KVX_EINVAL, c, 2, 1)
    refused(kvx.kvx_cache_inject_shared_stall, kvx.KVX_EINVAL, c, 1)


def test_rows_that_no_32_bits_count():
    """Up to 2^31 - 256 rows are shared; beyond, and rounding up to 256 of them passes 31 bits, each request reads its own."""
    c = kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16, n_q_heads=128)
    for n in (1 << 24, (1 << 24) - 1):
        assert kvx.kvx_cache_shared_bytes(c, n, 1) == 0
    kvx.kvx_cache_destroy(c)
