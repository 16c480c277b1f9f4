"""Rotations on the host: frequencies against their definition, and the refusals of the calls, none of which needs a GPU."""
import ctypes

import numpy as np
import pytest

import rotate_reference as ref
from test_decode_host import GEOM, LATENT, pool, refused

kvx = pytest.importorskip("disaggregated_prefill_decode_gb300.kvx")
A = 1 << 20                                                              # an address that is never read


@pytest.mark.parametrize("dim", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling=1, factor=4.0), dict(scaling=2, base=500000.0, factor=8.0, low=1.0, high=4.0, original=8192.0),
    dict(scaling=2, factor=32.0, low=2.0, high=2.5, original=1000.0), dict(scaling=3, factor=16.0, original=4096.0),
    dict(scaling=3, factor=1.0, original=4096.0), dict(scaling=3, factor=40.0, low=2.0, high=3.0, original=100.0, base=1000000.0)])
def test_frequencies(dim, kw):
    with kvx.kvx_rotation_create(dim=dim, **kw) as r:
        f, m = kvx.kvx_rotation_get(r)
    assert np.allclose(f, ref.frequencies(dim, **kw), rtol=1e-13, atol=0)
    assert m == (0.1 * np.log(kw["factor"]) + 1 if kw.get("scaling") == 3 else 1.0)


def test_magnitude_and_no_rotation():
    with kvx.kvx_rotation_create(dim=64, scaling=kvx.KVX_ROTATE_YARN, factor=8.0, original=4096.0, magnitude=0.75) as r:
        assert kvx.kvx_rotation_get(r)[1] == 0.75
    with kvx.kvx_rotation_create() as r:
        assert len(kvx.kvx_rotation_get(r)[0]) == 0


@pytest.mark.parametrize("status,kw", [
    ("EINVAL", dict(layout=2)), ("EINVAL", dict(layout=-1)), ("EINVAL", dict(scaling=4)), ("EINVAL", dict(scaling=-1)),
    ("EINVAL", dict(begin=-8)), ("EINVAL", dict(dim=-16)), ("EINVAL", dict(norm_dim=-8)), ("EINVAL", dict(base=1.0)),
    ("EINVAL", dict(base=-5.0)), ("EINVAL", dict(base=float("nan"))), ("EINVAL", dict(scaling=1)), ("EINVAL", dict(scaling=1, factor=0.5)),
    ("EINVAL", dict(scaling=2, factor=2.0)), ("EINVAL", dict(scaling=2, factor=2.0, low=4.0, high=4.0, original=100.0)),
    ("EINVAL", dict(scaling=2, factor=2.0, low=1.0, high=4.0)), ("EINVAL", dict(scaling=3, factor=2.0)),
    ("EINVAL", dict(scaling=3, factor=2.0, original=float("inf"))), ("EINVAL", dict(magnitude=-1.0)), ("EINVAL", dict(eps=-1e-6)),
    ("EINVAL", dict(eps=float("nan"))), ("EUNSUPPORTED", dict(dim=24)), ("EUNSUPPORTED", dict(dim=20, layout=1)),
    ("EUNSUPPORTED", dict(begin=4, dim=16)), ("EUNSUPPORTED", dict(norm_dim=12)), ("EUNSUPPORTED", dict(dim=272)),
])
def test_create_refusals(status, kw):
    refused(kvx.kvx_rotation_create, getattr(kvx, "KVX_" + status), **kw)


def test_handles():
    out = ctypes.c_void_p()
    cfg = kvx.kvx_rotation_config()
    cfg.reserved[1] = 1
    assert kvx._lib.kvx_rotation_create(ctypes.byref(cfg), ctypes.byref(out)) == kvx.KVX_EINVAL
    assert kvx._lib.kvx_rotation_create(None, ctypes.byref(out)) == kvx.KVX_EINVAL
    assert kvx._lib.kvx_rotation_create(ctypes.byref(kvx.kvx_rotation_config()), None) == kvx.KVX_EINVAL
    assert kvx._lib.kvx_rotation_destroy(None) == kvx.KVX_OK
    assert kvx._lib.kvx_rotation_get(None, None, 0, None, None) == kvx.KVX_EINVAL
    r = kvx.kvx_rotation_create(dim=64)
    assert kvx._lib.kvx_rotation_get(r.handle, None, 3, None, None) == kvx.KVX_EINVAL
    assert kvx._lib.kvx_rotation_get(r.handle, None, 0, None, None) == kvx.KVX_OK
    kvx.kvx_rotation_destroy(r)
    kvx.kvx_rotation_destroy(r)
    refused(kvx.kvx_rotation_get, kvx.KVX_EINVAL, r)


CALL = dict(layer=0, q=A, q_stride=256, q_weight=A, q_out=A + (1 << 16), q_out_stride=256, k=A, k_stride=128, k_weight=A, v=A, v_stride=128,
            positions=A, slots=A, n_tokens=3)


@pytest.mark.parametrize("bad", [
    dict(layer=2), dict(layer=-1), dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(k=None), dict(v=None), dict(slots=None),
    dict(positions=None), dict(q=None), dict(q_out=None), dict(q_stride=248), dict(q_out_stride=248), dict(k_stride=120),
    dict(v_stride=120), dict(k_stride=1 << 41), dict(q_stride=1 << 41), dict(q=A + 8), dict(q_out=A + 8), dict(q_weight=A + 8),
    dict(k_weight=A + 2), dict(k=A + 8), dict(v=A + 8), dict(q_stride=260), dict(q_out_stride=260), dict(k_stride=132), dict(v_stride=132),
    dict(slots=A + 4), dict(positions=A + 2), dict(q_out=A, q_out_stride=512)])
def test_call_refusals(bad):
    c = kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16, n_q_heads=4)
    with kvx.kvx_rotation_create(dim=64) as r:
        refused(kvx.kvx_cache_append_rotated, kvx.KVX_EINVAL, c, rotation=r, **{**CALL, **bad})


def test_rotations_of_other_heads_are_refused():
    c = kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16, n_q_heads=4)
    for kw in (dict(dim=80), dict(begin=16, dim=64), dict(dim=64, norm_dim=72)):
        with kvx.kvx_rotation_create(**kw) as r:
            refused(kvx.kvx_cache_append_rotated, kvx.KVX_EINVAL, c, rotation=r, **CALL)
    with kvx.kvx_rotation_create(dim=64) as r:
        kvx.kvx_cache_append_rotated(c, 0, r, None, 0, None, None, 0, None, 0, None, None, 0, None, None, 0)     # nothing to do
        latent = kvx.kvx_cache_create(pool(LATENT), value_type=kvx.KVX_E4M3, v_dim=512)
        refused(kvx.kvx_cache_append_rotated, kvx.KVX_EINVAL, latent, rotation=r, **{**CALL, "k_stride": 576, "q_stride": 576, "q_out_stride": 576})
        kvx.kvx_cache_destroy(c)
        refused(kvx.kvx_cache_append_rotated, kvx.KVX_EINVAL, c, rotation=r, **CALL)
    c = kvx.kvx_cache_create(pool(GEOM), value_type=kvx.KVX_BF16, n_q_heads=4)
    refused(kvx.kvx_cache_append_rotated, kvx.KVX_EINVAL, c, rotation=r, **CALL)


@pytest.mark.parametrize("kw", [dict(begin=2 ** 31 - 8, dim=16), dict(begin=2 ** 31 - 16, dim=16), dict(begin=2 ** 31 - 256, dim=256, layout=1),
                                dict(begin=584, dim=16), dict(begin=584), dict(norm_dim=2 ** 31 - 8), dict(norm_dim=584)])
def test_parts_beyond_the_widest_head_are_refused(kw):
    """begin + dim passes 31 bits: a sum that wrapped would be below any head's dim."""
    refused(kvx.kvx_rotation_create, kvx.KVX_EUNSUPPORTED, **kw)
