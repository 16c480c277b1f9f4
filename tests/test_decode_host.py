"""Refusals of the decode side's calls (kvx_slot_map, kvx_cache_*): every malformed argument is refused
before any CUDA call, so no GPU is needed; and calls with nothing to do return at once."""
import numpy as np
import pytest

import kvx_inputs

kvx = pytest.importorskip("disaggregated_prefill_decode_gb300.kvx")
PoolGeom = kvx_inputs.PoolGeom

GEOM = PoolGeom(2, 2, 1, 2, 64, 2, 16, 8)
LATENT = PoolGeom(1, 1, 1, 1, 576, 1, 64, 8)


def pool(geom, base=1 << 40, step=None):
    step = step or -(-geom.buffer_bytes // 256) * 256
    return kvx.Pool(geom, [base + i * step for i in range(geom.n_buffers)])


def refused(call, status, *args, **kw):
    with pytest.raises(kvx.KvxError) as ei:
        call(*args, **kw)
    assert ei.value.status == status, ei.value
    return str(ei.value)


@pytest.mark.parametrize("status,geom,kw", [
    ("EINVAL", GEOM, dict(value_type=0)),
    ("EINVAL", GEOM, dict(value_type=7)),
    ("EINVAL", GEOM, dict(value_type=3)),                                   # 8-bit values, 2-byte elements
    ("EINVAL", LATENT, dict(value_type=1)),
    ("EINVAL", GEOM, dict(value_type=1, io_type=2)),
    ("EINVAL", LATENT, dict(value_type=3, io_type=3)),
    ("EINVAL", GEOM, dict(value_type=1, n_q_heads=3)),
    ("EINVAL", GEOM, dict(value_type=1, n_q_heads=-2)),
    ("EINVAL", GEOM, dict(value_type=1, v_dim=32)),                         # two planes: v_dim is head_dim
    ("EINVAL", LATENT, dict(value_type=3, v_dim=577)),
    ("EINVAL", LATENT, dict(value_type=3, v_dim=-1)),
    ("EUNSUPPORTED", LATENT, dict(value_type=3, v_dim=500)),
    ("EINVAL", GEOM, dict(value_type=1, window=-1)),
    ("EINVAL", GEOM, dict(value_type=1, scale=float("nan"))),
    ("EINVAL", GEOM, dict(value_type=1, scale=-1.0)),
    ("EINVAL", GEOM, dict(value_type=1, k_scale=0.5)),
    ("EINVAL", LATENT, dict(value_type=3, v_dim=512, k_scale=0.5, v_scale=0.25)),
    ("EINVAL", LATENT, dict(value_type=3, v_dim=512, k_scale=1e-40)),
    ("EINVAL", LATENT, dict(value_type=3, v_dim=512, k_scale=float("inf"))),
    ("EUNSUPPORTED", GEOM.replace(n_planes=3), dict(value_type=1)),
    ("EUNSUPPORTED", GEOM.replace(n_shards=65), dict(value_type=1)),
    ("EUNSUPPORTED", GEOM.replace(head_dim=20), dict(value_type=1)),
    ("EUNSUPPORTED", GEOM.replace(head_dim=264), dict(value_type=1)),
    ("EUNSUPPORTED", LATENT.replace(head_dim=592), dict(value_type=3, v_dim=512)),
    ("EUNSUPPORTED", GEOM.replace(layout=2), dict(value_type=1)),
    ("EUNSUPPORTED", GEOM.replace(block_size=1 << 24, n_blocks=1), dict(value_type=1)),
    ("EINVAL", GEOM.replace(block_size=0), dict(value_type=1)),
])
def test_create_refusals(status, geom, kw):
    refused(kvx.kvx_cache_create, getattr(kvx, "KVX_" + status), pool(geom, step=1 << 32), **kw)


def test_create_refuses_unaligned_buffers_and_reserved_fields():
    refused(kvx.kvx_cache_create, kvx.KVX_EUNSUPPORTED, pool(GEOM, base=(1 << 40) + 8), value_type=1)
    import ctypes
    cfg = kvx.kvx_cache_config(1)
    cfg.reserved[2] = 1
    out = ctypes.c_void_p()
    p = pool(GEOM)
    assert kvx._lib.kvx_cache_create(ctypes.byref(p.struct), ctypes.byref(cfg), ctypes.byref(out)) == kvx.KVX_EINVAL
    assert kvx._lib.kvx_cache_create(ctypes.byref(p.struct), None, ctypes.byref(out)) == kvx.KVX_EINVAL
    assert kvx._lib.kvx_cache_create(None, ctypes.byref(kvx.kvx_cache_config(1)), ctypes.byref(out)) == kvx.KVX_EINVAL
    assert kvx._lib.kvx_cache_create(ctypes.byref(p.struct), ctypes.byref(kvx.kvx_cache_config(1)), None) == kvx.KVX_EINVAL


def test_destroy_twice_and_null():
    c = kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16)
    kvx.kvx_cache_destroy(c)
    kvx.kvx_cache_destroy(c)
    assert kvx._lib.kvx_cache_destroy(None) == kvx.KVX_OK
    refused(kvx.kvx_cache_append, kvx.KVX_EINVAL, c, 0, 16, 128, 16, 128, 16, 1)
    refused(kvx.kvx_cache_attend, kvx.KVX_EINVAL, c, 0, 16, 128, 16, 4, 4, 16, 1, 16, 128)
    refused(kvx.kvx_cache_status, kvx.KVX_EINVAL, c)


APPEND = dict(layer=0, k=1 << 20, k_stride=128, v=1 << 21, v_stride=128, slots=1 << 22, n_tokens=5)


@pytest.mark.parametrize("change", [dict(layer=-1), dict(layer=2), dict(k=None), dict(v=None), dict(slots=None), dict(n_tokens=-1),
                                    dict(n_tokens=1 << 31), dict(k_stride=127), dict(v_stride=120), dict(k_stride=132),
                                    dict(k=(1 << 20) + 8), dict(v=(1 << 21) + 2), dict(slots=(1 << 22) + 4),
                                    dict(k_stride=1 << 41)])
def test_append_refusals(change):
    with kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16) as c:
        refused(kvx.kvx_cache_append, kvx.KVX_EINVAL, c, **dict(APPEND, **change))
        kvx.kvx_cache_append(c, **dict(APPEND, n_tokens=0, k=None, v=None, slots=None))


def test_append_one_plane_takes_no_v():
    with kvx.kvx_cache_create(pool(LATENT), value_type=kvx.KVX_E4M3, v_dim=512) as c:
        refused(kvx.kvx_cache_append, kvx.KVX_EINVAL, c, 0, 1 << 20, 576, 1 << 21, 576, 1 << 22, 3)


ATTEND = dict(layer=0, q=1 << 20, q_stride=256, block_table=1 << 21, table_stride=4, max_blocks=4, seq_len=1 << 22, n_reqs=3,
              out=1 << 23, out_stride=256)


@pytest.mark.parametrize("change", [dict(layer=2), dict(q=None), dict(block_table=None), dict(seq_len=None), dict(out=None),
                                    dict(n_reqs=-1), dict(n_reqs=(1 << 24) + 1), dict(max_blocks=5), dict(max_blocks=-1),
                                    dict(q_stride=255), dict(out_stride=248), dict(q_stride=260), dict(q=(1 << 20) + 8),
                                    dict(out=(1 << 23) + 4), dict(out_stride=1 << 41), dict(seq_len=(1 << 22) + 2),
                                    dict(lse=(1 << 24) + 2)])
def test_attend_refusals(change):
    with kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16, n_q_heads=4) as c:
        refused(kvx.kvx_cache_attend, kvx.KVX_EINVAL, c, **dict(ATTEND, **change))
        kvx.kvx_cache_attend(c, **dict(ATTEND, n_reqs=0, q=None, block_table=None, seq_len=None, out=None))


def test_attend_refuses_values_above_512():
    with kvx.kvx_cache_create(pool(LATENT), value_type=kvx.KVX_E4M3) as c:
        refused(kvx.kvx_cache_attend, kvx.KVX_EUNSUPPORTED, c, **dict(ATTEND, q_stride=576, out_stride=576))


SLOTS = dict(ctx_len=1 << 20, new_len=1 << 21, n_reqs=3, block_size=16, free_blocks=1 << 22, n_free=4, block_table=1 << 23,
             table_stride=8, max_blocks=8, max_tokens=64, tok_off=1 << 24, slots=1 << 25, positions=None, seq_len=1 << 26,
             result=1 << 27)


@pytest.mark.parametrize("change", [dict(n_reqs=-1), dict(n_reqs=(1 << 24) + 1), dict(block_size=0), dict(n_free=-1),
                                    dict(max_blocks=9), dict(max_blocks=-1), dict(max_tokens=-1), dict(max_tokens=1 << 41),
                                    dict(ctx_len=None), dict(new_len=None), dict(seq_len=None), dict(tok_off=None),
                                    dict(result=None), dict(slots=None), dict(block_table=None), dict(free_blocks=None),
                                    dict(seq_len=1 << 20), dict(seq_len=1 << 21), dict(slots=(1 << 25) + 4),
                                    dict(positions=2), dict(tok_off=(1 << 24) + 4), dict(result=(1 << 27) + 1),
                                    dict(block_table=(1 << 23) + 2)])
def test_slot_map_refusals(change):
    refused(kvx.kvx_slot_map, kvx.KVX_EINVAL, **dict(SLOTS, **change))


def test_stall_hook_refusals():
    with kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16) as c:
        refused(kvx.kvx_cache_inject_stall, kvx.KVX_EUNSUPPORTED, c, 1)
    with kvx.kvx_cache_create(pool(LATENT), value_type=kvx.KVX_E4M3, v_dim=512) as c:
        refused(kvx.kvx_cache_inject_stall, kvx.KVX_EINVAL, c, 0)
        refused(kvx.kvx_cache_inject_stall, kvx.KVX_EINVAL, c, 5)
    refused(kvx.kvx_cache_inject_stall, kvx.KVX_EINVAL, c, 1)


@pytest.mark.parametrize("x", [3.7, "12", b"16", np.float32(8), np.float64(16), np.zeros(1, np.int64), np.array(16), [16], object()])
def test_pointers_are_tensors_or_integers(x):
    """What is neither is refused before the library sees an address made of it."""
    with pytest.raises(AttributeError):
        kvx._ptr(x)
    with kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16) as c:
        with pytest.raises(AttributeError):
            kvx.kvx_cache_append(c, **dict(APPEND, n_tokens=0, k=x))


def test_pointers_that_are_taken():
    assert kvx._ptr(None) == 0 and kvx._ptr(4096) == 4096 and kvx._ptr(np.int64(1 << 40)) == 1 << 40

    class Tensor:
        def data_ptr(self):
            return 512
    assert kvx._ptr(Tensor()) == 512
