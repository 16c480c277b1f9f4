"""GPU parity of the calls on pages through the C-ABI: tables, lists and pairs exactly, copies byte for byte."""
import numpy as np
import pytest

import kvx_inputs
import page_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
kvx = pytest.importorskip("disaggregated_prefill_decode_gb300.kvx")

PoolGeom = kvx_inputs.PoolGeom
NHD, HND = 0, 1


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(*shape, fill=-7, dtype=torch.int32):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


def batch(n, bs, hi, seed, shared=0, spare=1.3, width=None, idle=0.2):
    """A table whose rows share their first blocks, lengths, and the pool's size."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, hi + 1, n).astype(np.int32)
    lens[rng.random(n) < idle] = 0
    held = -(-lens // bs)
    width = width or max(int(held.max(initial=0)), 1) + 1
    n_blocks = int(spare * (held.sum() + shared)) + 3
    ids = rng.permutation(n_blocks).astype(np.int32)
    table = rng.integers(-5, n_blocks + 5, (n, width)).astype(np.int32)              # entries behind a row's blocks: anything
    at = shared
    for r in range(n):
        k = min(shared, held[r])
        table[r, :k] = ids[:k]
        table[r, k:held[r]] = ids[at:at + held[r] - k]
        at += held[r] - k
    return table, lens, n_blocks


def check_free(table, lens, bs, n_blocks, width=None, stride=None):
    width = table.shape[1] if width is None else width
    refs, free, result = ints(n_blocks + 1), ints(n_blocks + 1), ints(3, dtype=torch.int64)
    kvx.kvx_pages_free(dev(table), table.shape[1], width, dev(lens), len(lens), bs, n_blocks, refs, free, result)
    want = ref.free(table[:, :width], lens, bs, n_blocks)
    assert result.tolist() == want[2]
    assert np.array_equal(refs[:n_blocks].cpu().numpy(), want[0]) and refs[n_blocks] == -7
    k = len(want[1])
    assert np.array_equal(free[:k].cpu().numpy(), want[1]) and (free[k:] == -7).all()
    return want


@pytest.mark.parametrize("bs", [1, 16, 24])
@pytest.mark.parametrize("n,hi,shared", [(0, 0, 0), (1, 0, 0), (1, 1, 0), (3, 100, 2), (40, 700, 5), (300, 90, 1), (1500, 2000, 7),
                                         (17, 20000, 40)])
def test_free(n, hi, shared, bs):
    table, lens, n_blocks = batch(n, bs, hi, n + bs, shared)
    assert check_free(table, lens, bs, n_blocks)[2][2] == kvx.KVX_OK


def test_free_of_pools_of_any_size():
    for n_blocks in (0, 1, 31, 32, 33, 1023, 1024, 1025, 32768, 32769, 100001, 16 * 32768, 16 * 32768 + 1, 2000003):
        rng = np.random.default_rng(n_blocks)
        table = rng.integers(0, max(n_blocks, 1), (9, 700)).astype(np.int32)        # blocks held several times by one row, too
        lens = rng.integers(0, 700 * 8 + 1, 9).astype(np.int32) if n_blocks else np.zeros(9, np.int32)
        if n_blocks:
            table[0, 0], lens[0] = n_blocks - 1, max(lens[0], 1)
        assert check_free(table, lens, 8, n_blocks)[2][2] == kvx.KVX_OK


def test_free_out_of_range():
    table, lens, n_blocks = batch(50, 16, 400, 5, 3)
    for where, what in ((3, -1), (7, 2 ** 31 - 1), (9, -2 ** 31)):
        bad = lens.copy()
        bad[where] = what
        assert check_free(table, bad, 16, n_blocks)[2][2] == kvx.KVX_ERANGE
    hole = table.copy()
    hole[np.flatnonzero(lens > 20)[0], 1] = -1
    assert check_free(hole, lens, 16, n_blocks)[2][2] == kvx.KVX_ERANGE
    assert check_free(table, lens, 16, n_blocks // 2)[2][2] == kvx.KVX_ERANGE        # blocks beyond the pool
    assert check_free(table, lens, 16, n_blocks, width=3)[2][2] == kvx.KVX_ERANGE    # rows shorter than lengths
    assert check_free(table, lens, 16, n_blocks, width=0)[2][2] == kvx.KVX_ERANGE
    assert check_free(table, np.zeros_like(lens), 16, n_blocks, width=0)[2] == [0, n_blocks, kvx.KVX_OK]


def check_fork(table, lens, bs, parent, free_ids, stride=0):
    n_out, width = len(parent), table.shape[1]
    stride = stride or width
    new, new_len = ints(n_out + 1, stride), ints(n_out + 1)
    src, dst, result = ints(n_out + 1), ints(n_out + 1), ints(3, dtype=torch.int64)
    kvx.kvx_pages_fork(dev(table), width, width, dev(lens), len(lens), dev(parent), n_out, bs, dev(free_ids) if len(free_ids) else None,
                       len(free_ids), new, stride, new_len, src, dst, ints(len(lens) + 1), result)
    want = ref.fork(table, lens, bs, parent, free_ids)
    assert result.tolist() == want[4]
    assert np.array_equal(new[:n_out, :width].cpu().numpy(), want[0])
    assert (new[n_out] == -7).all() and (new[:, width:] == -7).all()
    assert new_len[:n_out].tolist() == want[1].tolist() and new_len[n_out] == -7
    assert src[:n_out].tolist() == want[2].tolist() and src[n_out] == -7
    assert dst[:n_out].tolist() == want[3].tolist() and dst[n_out] == -7
    return want[4][2]


@pytest.mark.parametrize("n,n_out", [(1, 0), (1, 1), (1, 40), (2, 3), (40, 40), (40, 7), (200, 1500), (3000, 2000), (5, 17000)])
@pytest.mark.parametrize("bs", [1, 16, 24])
def test_fork(n, n_out, bs):
    table, lens, _ = batch(n, bs, 200 if n_out > 5000 else 600, n + n_out + bs, 2)
    rng = np.random.default_rng(n_out)
    parent = rng.integers(-1, n, n_out).astype(np.int32)
    assert check_fork(table, lens, bs, parent, 100000 + rng.permutation(n_out + 1).astype(np.int32), stride=table.shape[1] + 5) == kvx.KVX_OK


def test_fork_keeps_rows_that_go_on():
    table, lens, _ = batch(100, 16, 500, 9)
    for parent in (np.arange(100), np.arange(100)[::-1], np.random.default_rng(1).permutation(100)):
        assert check_fork(table, lens, 16, parent.astype(np.int32), np.zeros(0, np.int32)) == kvx.KVX_OK       # no page is copied


def test_fork_out_of_range():
    table, lens, _ = batch(30, 16, 500, 11, idle=0)
    lens[lens % 16 == 0] += 1
    parent = (np.arange(60) // 2).astype(np.int32)
    for k in (0, 1, 29):
        assert check_fork(table, lens, 16, parent, np.arange(k, dtype=np.int32) + 1000) == kvx.KVX_ENOMEM
    some = parent.copy()
    some[[4, 9]] = (30, -2)
    assert check_fork(table, lens, 16, some, np.arange(60, dtype=np.int32)) == kvx.KVX_ERANGE
    bad = lens.copy()
    bad[[2, 5]] = (-3, 2 ** 31 - 1)
    assert check_fork(table, bad, 16, parent, np.arange(60, dtype=np.int32)) == kvx.KVX_ERANGE
    hole = table.copy()
    hole[7, (lens[7] - 1) // 16] = -1
    assert check_fork(hole, lens, 16, parent, np.arange(60, dtype=np.int32)) == kvx.KVX_ERANGE
    free = np.arange(60, dtype=np.int32)
    free[3] = -1
    assert check_fork(table, lens, 16, parent, free) == kvx.KVX_ERANGE
    assert check_fork(table[:0], lens[:0], 16, np.full(5, -1, np.int32), np.arange(9, dtype=np.int32)) == kvx.KVX_OK


def check_compact(table, lens, bs, n_blocks, max_moves=None, refs=None, in_place=False):
    refs = ref.free(table, lens, bs, n_blocks)[0] if refs is None else refs
    max_moves = n_blocks if max_moves is None else max_moves
    d_table = dev(table)
    new = d_table if in_place else ints(len(lens) + 1, table.shape[1])
    src, dst, result = ints(max_moves + 1), ints(max_moves + 1), ints(3, dtype=torch.int64)
    kvx.kvx_pages_compact(d_table, table.shape[1], table.shape[1], dev(lens), len(lens), bs, dev(refs), n_blocks, new, table.shape[1],
                          src, dst, max_moves, result)
    want = ref.compact(table, lens, bs, refs, max_moves)
    assert result.tolist() == want[2]
    assert np.array_equal(new[:len(lens)].cpu().numpy(), want[0])
    pairs = np.array(want[1], np.int32).reshape(-1, 2)
    k = len(pairs)
    assert src[:k].tolist() == pairs[:, 0].tolist() and dst[:k].tolist() == pairs[:, 1].tolist()
    assert (src[k:max_moves] == -1).all() and (dst[k:max_moves] == -1).all() and src[max_moves] == -7 and dst[max_moves] == -7
    assert in_place or (new[len(lens)] == -7).all()
    return want


@pytest.mark.parametrize("n,hi,shared", [(0, 0, 0), (1, 0, 0), (1, 30, 0), (3, 100, 2), (40, 700, 5), (300, 90, 1), (700, 2000, 7), (17, 20000, 40)])
@pytest.mark.parametrize("bs,spare", [(1, 3.0), (16, 1.0), (24, 1.7)])
def test_compact(n, hi, shared, bs, spare):
    table, lens, n_blocks = batch(n, bs, hi, n + bs, shared, spare)
    want = check_compact(table, lens, bs, n_blocks, in_place=n % 2 == 1)
    assert want[2][2] == kvx.KVX_OK
    if n_blocks:
        refs, free, _ = ref.free(want[0], lens, bs, n_blocks)
        assert free.tolist() == list(range(want[2][0], n_blocks))


def test_compact_of_large_pools():
    for n_blocks, held in ((1, 1), (1025, 1), (40000, 20000), (600000, 100), (1200000, 900000)):
        rng = np.random.default_rng(n_blocks)
        table = rng.permutation(n_blocks)[:held].astype(np.int32).reshape(1, -1)
        assert check_compact(table, np.array([held * 4], np.int32), 4, n_blocks)[2][2] == kvx.KVX_OK


def test_compact_out_of_range():
    table, lens, n_blocks = batch(60, 16, 900, 2, 3, 2.0)
    moves = check_compact(table, lens, 16, n_blocks)[2][1]
    assert check_compact(table, lens, 16, n_blocks, max_moves=moves)[2][2] == kvx.KVX_OK
    assert check_compact(table, lens, 16, n_blocks, max_moves=moves - 1)[2][2] == kvx.KVX_ENOMEM
    assert check_compact(table, lens, 16, n_blocks, max_moves=0, in_place=True)[2][2] == kvx.KVX_ENOMEM
    refs = ref.free(table, lens, 16, n_blocks)[0]
    refs[refs > 0] = np.random.default_rng(3).integers(0, 2, int((refs > 0).sum()))      # counts of another table
    assert check_compact(table, lens, 16, n_blocks, refs=refs)[2][2] == kvx.KVX_ERANGE
    bad = lens.copy()
    bad[4] = -1
    assert check_compact(table, bad, 16, n_blocks)[2][2] == kvx.KVX_ERANGE
    hole = table.copy()
    hole[np.flatnonzero(lens)[0], 0] = n_blocks + 7
    assert check_compact(hole, lens, 16, n_blocks)[2][2] == kvx.KVX_ERANGE


# ------------------------------------------------------------------------------------------------
# copies
# ------------------------------------------------------------------------------------------------

def pool_of(geom, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bufs = [torch.randint(0, 256, (geom.n_blocks, geom.block_size * geom.row_bytes), dtype=torch.uint8, device="cuda", generator=g)
            for _ in range(geom.n_buffers)]
    return bufs, kvx.Pool(geom, bufs)


@pytest.mark.parametrize("geom,kind,layers", [
    (PoolGeom(5, 2, 1, 2, 64, 2, 16, 40), 1, (0, 5)),
    (PoolGeom(5, 2, 3, 1, 8, 2, 1, 40), 2, (2, 4)),                       # blocks of one 16-byte vector
    (PoolGeom(2, 2, 2, 3, 48, 1, 5, 300, HND), 3, (0, 2)),
    (PoolGeom(3, 1, 1, 1, 576, 1, 64, 50), 3, (1, 3)),
    (PoolGeom(2, 2, 1, 8, 128, 2, 24, 30), 1, (1, 1)),
    (PoolGeom(1, 1, 1, 1, 16, 1, 1, 12000), 3, (0, 1)),
])
def test_copy(geom, kind, layers):
    bufs, pool = pool_of(geom, 3)
    rng = np.random.default_rng(4)
    order = rng.permutation(geom.n_blocks).astype(np.int32)
    n = geom.n_blocks // 3
    src, dst = order[:n], order[n:2 * n].copy()
    src = src[rng.integers(0, n, n)]                                        # one block may go to several places
    src = src.copy()
    none = rng.random(n) < 0.4
    src[none] = dst[none] = -1
    want = [b.cpu().numpy() for b in bufs]
    per = geom.n_planes * geom.n_shards
    for i in range(layers[0] * per, layers[1] * per):
        want[i][dst[~none]] = want[i][src[~none]]
    with kvx.kvx_cache_create(pool, kind, v_dim=0) as cache:
        kvx.kvx_cache_copy(cache, *layers, dev(src), dev(dst), n)
        assert kvx.kvx_cache_status(cache) == kvx.KVX_OK
        for a, b in zip(bufs, want):
            assert np.array_equal(a.cpu().numpy(), b)


def test_copy_reports_blocks_outside():
    geom = PoolGeom(2, 2, 1, 2, 64, 2, 16, 20)
    bufs, pool = pool_of(geom, 5)
    want = [b.cpu().numpy() for b in bufs]
    src, dst = np.array([1, 20, -1, 3, -5, 2 ** 31 - 1, 4], np.int32), np.array([9, 8, 7, -1, 6, 5, 10], np.int32)
    for w in want:
        w[[9, 10]] = w[[1, 4]]
    with kvx.kvx_cache_create(pool, kvx.KVX_BF16) as cache:
        kvx.kvx_cache_copy(cache, 0, 2, dev(src), dev(dst), 7)
        assert kvx.kvx_cache_status(cache) == kvx.KVX_ERANGE
        assert kvx.kvx_cache_status(cache) == kvx.KVX_OK
    for a, b in zip(bufs, want):
        assert np.array_equal(a.cpu().numpy(), b)


def test_copy_past_32_bits():
    """A buffer of 4.5 GiB: the offsets of its last blocks pass 32 bits."""
    geom = PoolGeom(1, 2, 1, 8, 128, 2, 16, 147456)
    big = torch.zeros(2, geom.n_blocks, 8192, dtype=torch.int32, device="cuda")     # 32 KiB a block
    big[0, 3], big[1, 3] = 11, 12
    big[0, 147455, 5], big[1, 147455, 5] = 13, 14
    with kvx.kvx_cache_create(kvx.Pool(geom, [big[0], big[1]]), kvx.KVX_BF16) as cache:
        kvx.kvx_cache_copy(cache, 0, 1, dev(np.array([3, 147455], np.int32)), dev(np.array([147454, 0], np.int32)), 2)
        assert kvx.kvx_cache_status(cache) == kvx.KVX_OK
    assert (big[0, 147454] == 11).all() and (big[1, 147454] == 12).all()
    assert big[0, 0, 5] == 13 and big[1, 0, 5] == 14 and big[0, 0].sum() == 13


def test_captured_step_of_pages():
    """Free, fork, copy and compact on a side stream, captured once and replayed on other tables."""
    bs, width, n = 16, 12, 6
    geom = PoolGeom(2, 2, 1, 2, 64, 2, bs, 200)
    bufs, pool = pool_of(geom, 6)
    side = torch.cuda.Stream()
    table, lens = ints(n, width, fill=-1), ints(n, fill=0)
    parent = ints(n)
    refs, free, r1 = ints(200), ints(200), ints(3, dtype=torch.int64)
    new, new_len, src, dst, scratch, r2 = ints(n, width), ints(n), ints(n), ints(n), ints(n), ints(3, dtype=torch.int64)
    with kvx.kvx_cache_create(pool, kvx.KVX_BF16) as cache:
        def step():
            kvx.kvx_pages_free(table, width, width, lens, n, bs, 200, refs, free, r1, side)
            kvx.kvx_pages_fork(table, width, width, lens, n, parent, n, bs, free, n, new, width, new_len, src, dst, scratch, r2, side)
            kvx.kvx_cache_copy(cache, 0, 2, src, dst, n, side)
        torch.cuda.synchronize()
        step()                                                                  # the handle's scratch
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for seed in (1, 2, 3):
            t, length, _ = batch(n, bs, 150, seed, 2, width=width, idle=0)
            p = np.random.default_rng(seed).integers(0, n, n).astype(np.int32)
            table.copy_(dev(t))
            lens.copy_(dev(length))
            parent.copy_(dev(p))
            before = [b.cpu().numpy() for b in bufs]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            want_refs, ids, res = ref.free(t, length, bs, 200)
            assert r1.tolist() == res and np.array_equal(refs.cpu().numpy(), want_refs)
            want = ref.fork(t, length, bs, p, ids[:n])
            assert r2.tolist() == want[4] and np.array_equal(new.cpu().numpy(), want[0])
            for a, b in zip(bufs, before):
                k = want[4][1]
                b[want[3][:k]] = b[want[2][:k]]
                assert np.array_equal(a.cpu().numpy(), b)
        assert kvx.kvx_cache_status(cache, side) == kvx.KVX_OK
