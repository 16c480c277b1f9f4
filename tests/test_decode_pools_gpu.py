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


@pytest.mark.parametrize("form", FORMS)
def test_layers_of_latents(form):
    """Each layer answers from its own buffers."""
    case = latents([300, 0, 1, 129], form)
    want, lse = case.run()
    layers = 3
    other = [torch.zeros_like(b) for b in case.bufs]
    for at in range(layers):
        bufs = sum([case.bufs if i == at else other for i in range(layers)], [])
        with create(case, case.geom.replace(n_layers=layers), bufs) as c:
            assert torch.equal(attend(case, c, layer=at), want)
            out = attend(case, c, layer=(at + 1) % layers)
            assert (out == 0).all()                                        # values of 0
            x = torch.randn((1, case.heads, 576), device="cuda").to(case.iodtype)
            before = [b.clone() for b in bufs]
            slot = int(case.table[0, 1]) * 64 + 7
            kvx.kvx_cache_append(c, at, x, case.heads * 576, None, 0, dev(np.array([slot], np.int64)), 1)
            assert kvx.kvx_cache_status(c) == kvx.KVX_OK
            shards = case.geom.n_shards
            for i, (a, b) in enumerate(zip(bufs, before)):
                assert torch.equal(a, b) == (i // shards != at)
            for a, b in zip(case.bufs, before[at * shards:]):
                a.copy_(b)


@pytest.mark.parametrize("form", FORMS)
def test_latents_in_a_capture(form):
    """Slot map, append and attention of a step in one graph; the second replay sees lengths of its own."""
    case = latents([900, 64, 5], form)
    case.run()
    n, heads, hq = 3, case.heads, case.heads * case.group
    bufs = [b.clone() for b in case.bufs]
    spare = [b for b in range(case.geom.n_blocks) if b not in set(case.table[r, j] for r, k in enumerate(case.lens) for j in range(-(-k // 64)))]
    free = dev(np.array(spare, np.int32))
    table = case.d_table.clone()
    x = torch.randn((n, heads, 576), device="cuda").to(case.iodtype)
    ctx, new = dev(np.array(case.lens, np.int32)), torch.ones(n, dtype=torch.int32, device="cuda")
    seq, tok_off = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    slots, result = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    out = torch.zeros((n, hq, 512), dtype=case.iodtype, device="cuda")
    lse = torch.zeros((n, hq), dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()

    def step(c):
        kvx.kvx_slot_map(ctx, new, n, 64, free, len(free), table, table.shape[1], case.width, n, tok_off, slots, None, seq, result, side)
        kvx.kvx_cache_append(c, 0, x, heads * 576, None, 0, slots, n, side)
        kvx.kvx_cache_attend(c, 0, case.d_q, hq * 576, table, table.shape[1], case.width, seq, n, out, hq * 512, lse, side)

    with create(case, case.geom, bufs) as c:
        step(c)                                                            # allocates
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(c)
        for i, lens in enumerate((case.lens, [700, 63, 0], [899, 0, 4])):
            ctx.copy_(dev(np.array(lens, np.int32)))
            table.copy_(case.d_table)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert result[2].item() == kvx.KVX_OK
            got = out.clone(), lse.clone()
            table.copy_(case.d_table)
            with torch.cuda.stream(side):
                step(c)
            torch.cuda.synchronize()
            assert torch.equal(got[0], out) and torch.equal(got[1], lse)
            if i == 0:                                                     # later steps write slots that were live here
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert kvx.kvx_cache_status(c) == kvx.KVX_OK


@pytest.mark.parametrize("form", [("bf16", 16, 1), ("e4m3", 16, 1), ("e4m3", 40, 1), ("e4m3", 16, 2)])
def test_latents_beyond_4_gib(form):
    """Rows past 2^32 bytes of a buffer."""
    small = latents([500, 70], form)
    want, lse = small.run()
    esz = small.geom.elem_bytes
    size = 64 * 576 * esz
    n_blocks = (1 << 32) // size + 2000
    geom = small.geom.replace(n_blocks=n_blocks)
    bufs = [torch.zeros(geom.buffer_bytes, dtype=torch.uint8, device="cuda") for _ in small.bufs]
    used = [8, 2]
    far = np.full(small.table.shape, -1, np.int32)
    at = n_blocks - 1
    for r, k in enumerate(used):
        for j in range(k):
            far[r, j] = at
            for b, s in zip(bufs, small.bufs):
                b[at * size:][:size] = s[int(small.table[r, j]) * size:][:size]
            at -= 1
    assert at * size > 1 << 32
    with create(small, geom, bufs) as c:
        assert torch.equal(attend(small, c, table=dev(far)), want)
        x = torch.randn((2, small.heads, 576), device="cuda").to(small.iodtype)
        last = n_blocks * 64 - 1
        kvx.kvx_cache_append(c, 0, x, small.heads * 576, None, 0, dev(np.array([last, 1], np.int64)), 2)
        assert kvx.kvx_cache_status(c) == kvx.KVX_OK
        for b in bufs:
            rows = b.view(-1, 576 * esz)
            assert rows[last].any() and rows[1].any() and not rows[0].any() and not rows[2].any()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("at", [0, 77, 699])
def test_nan_in_a_live_latent(form, at):
    """A NaN key makes its request NaN, every head of its shard, and no other; so does a NaN in an element of the value."""
    for element in (3, 570):
        case = latents([700, 20, 300], form)
        want, lse = case.run()
        view = typed(case.bufs[0], case.geom, TYPES[case.value][1])
        raw = view.view(torch.uint8 if case.geom.elem_bytes == 1 else torch.int16)
        raw[int(case.table[0, at // 64]), at % 64, 0, element] = 0x7F if case.geom.elem_bytes == 1 else 0x7FFF
        out, got = case.run()
        assert torch.isnan(out[0, :case.group]).all() and torch.isnan(got[0, :case.group]).all()
        assert torch.equal(out[0, case.group:], want[0, case.group:]) and torch.equal(out[1:], want[1:]) and torch.equal(got[1:], lse[1:])


@pytest.mark.parametrize("layout", [NHD, HND])
@pytest.mark.parametrize("form", FORMS)
def test_what_lies_outside_the_window_or_the_length_is_not_seen(form, layout):
    """NaN and infinities in cached positions before the window, in slots after the length, and in blocks of no request."""
    case = latents([700, 20, 300], form, window=130, layout=layout)
    want, lse = case.run()
    dtype = TYPES[case.value][1]
    for b in case.bufs:
        view = typed(b, case.geom, dtype)
        for r, n in enumerate(case.lens):
            for t in range(max(0, n - 130)):
                view[int(case.table[r, t // 64]), t % 64] = float("nan") if t % 2 or case.value == "e4m3" else float("inf")
    out, got = case.run()
    assert torch.equal(out, want) and torch.equal(got, lse)
    case.check(out, got)
