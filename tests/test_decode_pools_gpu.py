"""Pools of latents beside the plain one: several layers, buffers in different memory, buffers past 4 GiB, NaN, captures."""
import numpy as np
import pytest

from test_decode_gpu import HND, NHD, TYPES, Attend, PoolGeom, dev, kvx, pinned, torch, typed

pytestmark = pytest.mark.gpu

# shards 1: the kernel of tensor maps; 2: that of warp products
FORMS = [("bf16", 16, 1), ("f16", 24, 1), ("e4m3", 16, 1), ("e4m3", 40, 1), ("bf16", 5, 2), ("e4m3", 16, 2)]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def latents(lens, form, **kw):
    value, group, shards = form
    return Attend(lens, value=value, planes=1, shards=shards, hps=1, group=group, dim=576, v_dim=512, bs=64, **kw)


def create(case, geom, bufs):
    scale = 0.03 if case.value == "e4m3" else 0.0
    return kvx.kvx_cache_create(kvx.Pool(geom, bufs), TYPES[case.value][0], n_q_heads=case.heads * case.group, v_dim=case.v_dim, k_scale=scale)


def attend(case, cache, layer=0, table=None, stream=None):
    n, hq = len(case.lens), case.heads * case.group
    out = torch.zeros((n, hq, case.v_dim), dtype=case.iodtype, device="cuda")
    table = case.d_table if table is None else table
    torch.cuda.synchronize()
    kvx.kvx_cache_attend(cache, layer, case.d_q, hq * case.dim, table, table.shape[1], case.width, case.d_len, n, out, hq * case.v_dim,
                         None, stream)
    return out


def test_a_latent_layer_in_host_memory_is_refused():
    """Whichever layer it is: the first and the last buffer do not speak for those between."""
    for layer in range(3):
        case = latents([100, 3], ("bf16", 16, 1))
        case.run()
        bufs = [case.bufs[0], case.bufs[0].clone(), case.bufs[0].clone()]
        host = pinned([case.bufs[0]])
        bufs[layer] = host[0]
        with create(case, case.geom.replace(n_layers=3), bufs) as c:
            with pytest.raises(kvx.KvxError) as ei:
                attend(case, c, layer=0)
            assert ei.value.status == kvx.KVX_EUNSUPPORTED


@pytest.mark.parametrize("form", FORMS + [("bf16", 4, 0), ("e4m3", 12, 0)])
def test_a_pool_without_blocks(form):
    """It may have no memory either. Every cached position is out of bounds: reported, outputs 0, and appends skip."""
    value, group, shards = form
    planes, dim, v_dim = (1, 576, 512) if shards else (2, 128, 128)
    case = Attend([0, 70, 3], value=value, planes=planes, shards=max(shards, 1), hps=1, group=group, dim=dim, v_dim=v_dim, bs=64)
    case.run()
    n, heads = 3, max(shards, 1)
    geom = case.geom.replace(n_blocks=0)
    with create(case, geom, [None] * geom.n_buffers) as c:
        out = attend(case, c)
        assert (out == 0).all()
        assert kvx.kvx_cache_status(c) == kvx.KVX_ERANGE
        x = torch.zeros((n, heads, dim), dtype=case.iodtype, device="cuda")
        kvx.kvx_cache_append(c, 0, x, heads * dim, x if planes == 2 else None, heads * dim, dev(np.array([0, -1, 5], np.int64)), n)
        assert kvx.kvx_cache_status(c) == kvx.KVX_ERANGE and "2 slots" in kvx.kvx_last_error()
