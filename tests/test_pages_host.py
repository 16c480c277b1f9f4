"""Refusals of the calls on pages: every malformed argument is refused before any CUDA call, so no GPU is needed."""
import pytest

from test_decode_host import GEOM, pool, refused

kvx = pytest.importorskip("disaggregated_prefill_decode_gb300.kvx")
T, L, P, R = 1 << 20, 1 << 21, 1 << 22, 1 << 23                           # addresses that are never read

FREE = dict(block_table=T, table_stride=8, max_blocks=8, seq_len=L, n_reqs=4, block_size=16, n_blocks=100, refs=P, free_blocks=P + 4096,
            result=R)
FORK = dict(block_table=T, table_stride=8, max_blocks=8, seq_len=L, n_reqs=4, parent=P, n_out=6, block_size=16, free_blocks=P + 64,
            n_free=5, new_table=P + 4096, new_stride=8, new_len=P + 8192, src_blocks=P + 8256, dst_blocks=P + 8320, scratch=P + 8384,
            result=R)
COMPACT = dict(block_table=T, table_stride=8, max_blocks=8, seq_len=L, n_reqs=4, block_size=16, refs=P, n_blocks=100, new_table=P + 4096,
               new_stride=8, src_blocks=P + 8192, dst_blocks=P + 12288, max_moves=9, result=R)
TABLE = [dict(n_reqs=-1), dict(n_reqs=(1 << 24) + 1), dict(block_size=0), dict(block_size=-4), dict(max_blocks=-1),
         dict(table_stride=7), dict(table_stride=(1 << 36) + 1), dict(block_table=None), dict(seq_len=None), dict(block_table=T + 2),
         dict(seq_len=L + 1), dict(result=None), dict(result=R + 4)]


@pytest.mark.parametrize("bad", TABLE + [dict(n_blocks=-1), dict(n_blocks=1 << 31), dict(refs=None), dict(free_blocks=None),
                                         dict(refs=P + 2), dict(free_blocks=P + 1)])
def test_free_refusals(bad):
    refused(kvx.kvx_pages_free, kvx.KVX_EINVAL, **{**FREE, **bad})


@pytest.mark.parametrize("bad", TABLE + [
    dict(n_out=-1), dict(n_out=(1 << 24) + 1), dict(n_free=-1), dict(free_blocks=None), dict(new_stride=7), dict(new_table=None),
    dict(new_len=None), dict(src_blocks=None), dict(dst_blocks=None), dict(scratch=None), dict(parent=None), dict(parent=P + 2),
    dict(new_table=P + 2), dict(scratch=P + 1), dict(new_table=T), dict(new_table=T + 4 * (3 * 8 + 7)), dict(new_len=L),
    dict(new_len=L + 12), dict(new_table=T - 4 * (5 * 8 + 7))])
def test_fork_refusals(bad):
    refused(kvx.kvx_pages_fork, kvx.KVX_EINVAL, **{**FORK, **bad})


@pytest.mark.parametrize("bad", TABLE + [
    dict(n_blocks=-1), dict(n_blocks=1 << 31), dict(refs=None), dict(max_moves=-1), dict(max_moves=1 << 31), dict(src_blocks=None),
    dict(dst_blocks=None), dict(new_table=None), dict(new_stride=7), dict(new_table=T + 4), dict(new_table=T, new_stride=9),
    dict(refs=P + 2), dict(new_table=P + 4098)])
def test_compact_refusals(bad):
    refused(kvx.kvx_pages_compact, kvx.KVX_EINVAL, **{**COMPACT, **bad})


def test_copy_refusals():
    c = kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16)
    for bad in (dict(layer_begin=-1), dict(layer_begin=2, layer_end=1), dict(layer_end=3), dict(n_pairs=-1), dict(src_blocks=None),
                dict(dst_blocks=None), dict(src_blocks=P + 2), dict(dst_blocks=P + 1)):
        refused(kvx.kvx_cache_copy, kvx.KVX_EINVAL, c, **{**dict(layer_begin=0, layer_end=2, src_blocks=P, dst_blocks=P, n_pairs=3), **bad})
    kvx.kvx_cache_copy(c, 0, 2, None, None, 0)                             # nothing to do, no CUDA call
    kvx.kvx_cache_copy(c, 1, 1, P, P, 5)
    kvx.kvx_cache_destroy(c)
    refused(kvx.kvx_cache_copy, kvx.KVX_EINVAL, c, 0, 1, P, P, 1)
