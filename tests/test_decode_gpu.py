"""GPU parity of the decode side through the C-ABI: slot maps and appends exactly, attention within the
bounds its arithmetic allows of a plain 64-bit statement (tests/decode_reference.py)."""
import numpy as np
import pytest

import decode_reference as ref
import kvx_inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
kvx = pytest.importorskip("disaggregated_prefill_decode_gb300.kvx")

PoolGeom = kvx_inputs.PoolGeom
NHD, HND = 0, 1
TYPES = {"bf16": (1, torch.bfloat16, 2), "f16": (2, torch.float16, 2), "e4m3": (3, torch.float8_e4m3fn, 1)}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------------------------------------
# slot maps
# ------------------------------------------------------------------------------------------------

def check_slot_map(ctx, new, bs, free, table, max_blocks, max_tokens, positions=True, shift=0):
    want = ref.slot_map(ctx, new, bs, free, table, max_blocks, max_tokens)
    n = len(ctx)
    d_table = dev(table)
    tok_off = torch.full((n + 1,), -7, dtype=torch.int64, device="cuda")
    slots = torch.full((max_tokens + 1 + shift,), -9, dtype=torch.int64, device="cuda")
    pos = torch.full((max_tokens + 1,), -9, dtype=torch.int32, device="cuda") if positions else None
    seq = torch.full((max(n, 1),), -7, dtype=torch.int32, device="cuda")
    result = torch.full((3,), -7, dtype=torch.int64, device="cuda")
    kvx.kvx_slot_map(dev(ctx), dev(new), n, bs, dev(free) if len(free) else None, len(free), d_table, table.shape[1], max_blocks,
                     max_tokens, tok_off, slots[shift:], pos, seq, result)
    assert result.tolist() == [want[5], want[6], want[7]]
    assert tok_off.tolist() == want[0].tolist()
    assert np.array_equal(slots[shift:shift + max_tokens].cpu().numpy(), want[1])
    assert slots[-1].item() == -9 and (not shift or slots[0].item() == -9)
    if positions:
        k = len(want[2])
        assert np.array_equal(pos[:k].cpu().numpy(), want[2])
        assert (pos[k:] == -9).all()
    assert seq[:n].tolist() == want[3].tolist()
    assert np.array_equal(d_table.cpu().numpy(), want[4])
    return want[7]


def slot_inputs(n, bs, ctx_hi, new_hi, seed, spare=3, width=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, n).astype(np.int32)
    new = rng.integers(0, new_hi + 1, n).astype(np.int32)
    ctx[rng.random(n) < 0.2] = 0
    new[rng.random(n) < 0.2] = 0
    had, need = -(-ctx // bs), -(-(ctx + new) // bs)
    width = width or max(int(need.max(initial=0)), 1) + 2
    ids = rng.permutation(int(need.sum()) + spare).astype(np.int32)
    table = np.full((n, width), -1, np.int32)
    at = 0
    for r in range(n):
        table[r, :had[r]] = ids[at:at + had[r]]
        at += had[r]
    return ctx, new, ids[at:], table


@pytest.mark.parametrize("bs", [1, 16, 24, 64])
@pytest.mark.parametrize("n,ctx_hi,new_hi", [(0, 0, 0), (1, 0, 1), (1, 50, 700), (5, 100, 1), (33, 300, 3), (300, 90, 40),
                                             (1024, 40, 2), (1025, 40, 1), (3000, 20, 5), (7, 10, 9000)])
def test_slot_map(n, ctx_hi, new_hi, bs):
    ctx, new, free, table = slot_inputs(n, bs, ctx_hi, new_hi, n + bs)
    assert check_slot_map(ctx, new, bs, free, table, table.shape[1], int(new.sum())) == kvx.KVX_OK


@pytest.mark.parametrize("positions,shift,tail", [(False, 0, 0), (True, 1, 5), (True, 0, 3001), (False, 1, 1)])
def test_slot_map_tail_alignment_and_no_positions(positions, shift, tail):
    ctx, new, free, table = slot_inputs(40, 16, 100, 60, 3)
    assert check_slot_map(ctx, new, 16, free, table, table.shape[1], int(new.sum()) + tail, positions, shift) == kvx.KVX_OK


def test_slot_map_out_of_range():
    ctx, new, free, table = slot_inputs(50, 16, 200, 90, 4)
    total, width = int(new.sum()), table.shape[1]
    assert check_slot_map(ctx, new, 16, free[:7], table, width, total) == kvx.KVX_ENOMEM
    assert check_slot_map(ctx, new, 16, free[:0], table, width, total) == kvx.KVX_ENOMEM
    assert check_slot_map(ctx, new, 16, free, table, width - 5, total) == kvx.KVX_ERANGE     # rows too short
    assert check_slot_map(ctx, new, 16, free, table, 0, total) == kvx.KVX_ERANGE
    assert check_slot_map(ctx, new, 16, free, table, width, total - 11) == kvx.KVX_ERANGE    # tokens beyond max_tokens
    assert check_slot_map(ctx, new, 16, free, table, width, 0) == kvx.KVX_ERANGE
    bad = new.copy()
    bad[::7] = -5
    assert check_slot_map(ctx, bad, 16, free, table, width, total) == kvx.KVX_ERANGE
    bad = ctx.copy()
    bad[3] = -2 ** 31
    assert check_slot_map(bad, new, 16, free, table, width, total) in (kvx.KVX_ERANGE, kvx.KVX_ENOMEM)
    hole = table.copy()                                                     # a request that goes on in a block it lacks
    ctx[9], new[9] = 17, 4
    hole[9] = -1
    hole[9, 0] = 0
    assert check_slot_map(ctx, new, 16, np.arange(1000, 2000, dtype=np.int32), hole, width, total + 90) == kvx.KVX_ERANGE


@pytest.mark.parametrize("n,max_tokens", [(1025, 1000), (2048, 1000), (2049, 1000), (3000, 1000), (1025, 999), (2100, 900), (1024, 999),
                                          (1025, 0), (2100, 1255)])
def test_slot_map_passes_without_tokens(n, max_tokens):
    """1000 tokens, no multiple of a tile's, in the first 1024 requests; those after them, other passes of the kernel, idle or
    with all their tokens beyond max_tokens."""
    ctx, new = np.arange(n, dtype=np.int32) % 23, np.zeros(n, np.int32)
    new[:1000] = 1
    if max_tokens < 1000:
        new[1024:] = 2
    table = np.full((n, 4), -1, np.int32)
    had = -(-ctx // 8)
    table[np.arange(4) < had[:, None]] = np.arange(had.sum())
    free = (int(had.sum()) + np.arange(n)).astype(np.int32)
    status = check_slot_map(ctx, new, 8, free, table, 4, max_tokens)
    assert status == (kvx.KVX_ERANGE if new.sum() > max_tokens else kvx.KVX_OK)


# ------------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------------

def make_pool(geom, dtype, seed, align=512, big=None):
    """Random bytes in every buffer, NaN codes among them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    per = -(-geom.buffer_bytes // align) * align
    mem = torch.randint(0, 256, (max(per * geom.n_buffers, align),), dtype=torch.uint8, device="cuda", generator=g)
    return [mem[i * per:i * per + geom.buffer_bytes] for i in range(geom.n_buffers)]


def typed(buf, geom, dtype):
    """[block][slot][head][dim] view of a buffer, whatever its layout."""
    if geom.layout == NHD:
        return buf.view(dtype).view(geom.n_blocks, geom.block_size, geom.heads_per_shard, geom.head_dim)
    return buf.view(dtype).view(geom.n_blocks, geom.heads_per_shard, geom.block_size, geom.head_dim).transpose(1, 2)


@pytest.mark.parametrize("layout", [NHD, HND])
@pytest.mark.parametrize("value,io,planes,shards,hps,dim,bs", [
    ("bf16", "bf16", 2, 1, 2, 64, 16), ("f16", "f16", 2, 4, 2, 128, 16), ("bf16", "bf16", 2, 1, 17, 128, 20),
    ("e4m3", "bf16", 1, 1, 1, 576, 64), ("e4m3", "f16", 2, 2, 3, 80, 1), ("bf16", "bf16", 1, 1, 1, 24, 8)])
@pytest.mark.parametrize("n", [1, 37, 2600])
def test_append(value, io, planes, shards, hps, dim, bs, layout, n):
    vt, vdtype, esz = TYPES[value]
    iot, iodtype, _ = TYPES[io]
    heads = shards * hps
    geom = PoolGeom(2, planes, shards, hps, dim, esz, bs, -(-n // bs) + 9, layout)
    bufs = make_pool(geom, vdtype, 1)
    before = [b.clone() for b in bufs]
    rng = np.random.default_rng(n)
    slots = rng.permutation(geom.n_blocks * bs)[:n].astype(np.int64)
    skip = rng.random(n) < 0.1
    slots[skip] = -1
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    both = torch.randn((n, 3, heads, dim), device="cuda", generator=g).to(iodtype)     # q between: strides of their own
    both[0, 0, 0, :4] = torch.tensor([float("nan"), float("inf"), -1e4, 0.0], device="cuda").to(iodtype)
    scale = 0.037 if value == "e4m3" else 0.0
    with kvx.kvx_cache_create(kvx.Pool(geom, bufs), vt, iot, k_scale=scale, v_scale=scale) as c:
        kvx.kvx_cache_append(c, 1, both[:, 0], 3 * heads * dim, both[:, 2] if planes == 2 else None, 3 * heads * dim, dev(slots), n)
        assert kvx.kvx_cache_status(c) == kvx.KVX_OK
    inverse = float(np.float32(1.0) / np.float32(scale)) if scale else 1.0
    at = dev(slots[~skip])
    for p in range(planes):
        x = both[:, 2 * p][dev(~skip)]
        if value == "e4m3":
            x = (x.float() * inverse).clamp(-448, 448).to(vdtype)
        for s in range(shards):
            i = (planes + p) * shards + s
            view = typed(before[i], geom, vdtype).view(torch.uint8 if esz == 1 else torch.int16)
            view[at // bs, at % bs] = x[:, s * hps:(s + 1) * hps].contiguous().view(view.dtype)
    for i, (a, b) in enumerate(zip(bufs, before)):
        if value == "e4m3":                                                 # NaN has two codes: either
            a, b = (torch.where(t & 0x7F == 0x7F, 0x7F, t) for t in (a, b))
        assert torch.equal(a, b), i


def test_append_reports_slots_outside_the_pool():
    geom = PoolGeom(1, 2, 1, 2, 64, 2, 16, 4)
    bufs = make_pool(geom, torch.bfloat16, 3)
    before = [b.clone() for b in bufs]
    x = torch.randn((4, 2, 64), device="cuda").to(torch.bfloat16)
    with kvx.kvx_cache_create(kvx.Pool(geom, bufs), kvx.KVX_BF16) as c:
        kvx.kvx_cache_append(c, 0, x, 128, x, 128, dev(np.array([64, -2, 2 ** 40, -1], np.int64)), 4)
        assert kvx.kvx_cache_status(c) == kvx.KVX_ERANGE
        assert "3 slots" in kvx.kvx_last_error()
        assert kvx.kvx_cache_status(c) == kvx.KVX_OK
    assert all(torch.equal(a, b) for a, b in zip(bufs, before))


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------

P_UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -11}        # weights rounded to the type of the products


class Attend:
    """A pool of one layer whose unused slots hold NaN, a table with garbage past its use, queries, and the 64-bit answer."""

    def __init__(self, lens, value="bf16", io=None, planes=2, shards=1, hps=2, group=4, dim=64, v_dim=0, bs=16, layout=NHD, window=0,
                 scale=0.0, seed=0, k_scale=0.03, v_scale=0.05, extra_blocks=5, spread=1.0):
        self.value, self.io = value, io or (value if value != "e4m3" else "bf16")
        vt, vdtype, esz = TYPES[value]
        iot, iodtype, _ = TYPES[self.io]
        self.lens, self.bs, self.group, self.heads = list(lens), bs, group, shards * hps
        rng = np.random.default_rng(seed)
        need = [-(-n // bs) for n in lens]
        self.geom = geom = PoolGeom(1, planes, shards, hps, dim, esz, bs, sum(need) + extra_blocks, layout)
        order = rng.permutation(geom.n_blocks)
        self.width = max(need + [1]) + 1
        self.table = np.full((len(lens), self.width + 2), 2 ** 30, np.int32)
        at = 0
        for r, k in enumerate(need):
            self.table[r, :k] = order[at:at + k]
            at += k
        scales = (k_scale, k_scale if planes == 1 else v_scale) if value == "e4m3" else (0.0, 0.0)
        self.bufs = []
        self.host = []                                                     # per plane: [row][head][dim] float64, scaled
        for p in range(planes):
            parts = []
            for s in range(shards):
                buf = torch.full((max(geom.buffer_bytes, 16),), 0xFF, dtype=torch.uint8, device="cuda")[:geom.buffer_bytes]
                view = typed(buf, geom, vdtype)
                x = torch.from_numpy(rng.standard_normal(tuple(view.shape)).astype(np.float32) * spread)
                x = (x / scales[p]).clamp(-448, 448).to(vdtype) if esz == 1 else x.to(vdtype)
                raw = view.view(torch.uint8 if esz == 1 else torch.int16)
                used = torch.zeros((geom.n_blocks, bs), dtype=torch.bool)
                for r, n in enumerate(lens):
                    for j in range(need[r]):
                        used[int(self.table[r, j]), :min(bs, n - j * bs)] = True
                raw[used.cuda()] = x.view(raw.dtype)[used].cuda()
                self.bufs.append(buf)
                parts.append(x.double().numpy().reshape(geom.n_blocks * bs, hps, dim) * (scales[p] or 1.0))
            self.host.append(np.concatenate(parts, 1))
        self.q = torch.from_numpy(rng.standard_normal((len(lens), self.heads * group, dim)).astype(np.float32)).to(iodtype)
        self.dim, self.v_dim, self.window = dim, v_dim or dim, window
        self.scale = scale or 1 / np.sqrt(dim)
        self.cache = kvx.kvx_cache_create(kvx.Pool(geom, self.bufs), vt, iot, n_q_heads=self.heads * group, v_dim=v_dim,
                                          window=window, scale=scale, k_scale=scales[0], v_scale=scales[1])
        self.iodtype = iodtype

    def run(self, stream=None, pad=0, lse=True):
        n, hq = len(self.lens), self.heads * self.group
        q = torch.zeros((n, hq * self.dim + pad), dtype=self.iodtype)
        q[:, :hq * self.dim] = self.q.reshape(n, -1)
        self.d_q, self.d_table, self.d_len = q.cuda(), dev(self.table), dev(np.array(self.lens, np.int32))
        out = torch.full((n, hq * self.v_dim + pad), 7.0, dtype=self.iodtype, device="cuda")
        self.d_lse = torch.full((n, hq), 7.0, dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        kvx.kvx_cache_attend(self.cache, 0, self.d_q, q.shape[1], self.d_table, self.table.shape[1], self.width, self.d_len, n, out,
                             out.shape[1], self.d_lse if lse else None, stream)
        torch.cuda.synchronize()
        if pad:
            assert (out[:, hq * self.v_dim:] == 7.0).all()
        return out[:, :hq * self.v_dim].reshape(n, hq, self.v_dim).clone(), self.d_lse

    def check(self, out, lse, table=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        table = self.table if table is None else table
        for r, n in enumerate(self.lens):
            first = max(0, n - self.window) if self.window else 0
            rows = ref.rows_of(table[r], np.arange(first, max(n, 0)), self.bs, self.geom.n_blocks)
            for h in range(self.heads):
                hs = slice(h * self.group, (h + 1) * self.group)
                k, v = self.host[0][rows, h], self.host[-1][rows, h, :self.v_dim]
                o, l, weight, spread, floor = ref.attend(self.q[r, hs].double().numpy(), k, v, self.scale)
                b_out, b_lse = ref.attend_bounds(o, l, weight, spread, floor, self.dim, len(rows), self.io, P_UNIT[self.value])
                if len(rows) == 0:
                    assert (out[r, hs] == 0).all() and (lse[r, hs] == -np.inf).all(), (r, h)
                    continue
                bad = np.abs(out[r, hs] - o) - b_out
                assert np.isfinite(out[r, hs]).all() and (bad <= 0).all(), (r, h, n, bad.max())
                assert (np.abs(lse[r, hs] - l) <= b_lse).all(), (r, h, n, np.abs(lse[r, hs] - l).max())


def check_attend(lens, **kw):
    case = Attend(lens, **kw)
    case.check(*case.run())
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    kvx.kvx_cache_destroy(case.cache)


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257, 0, 511]


@pytest.mark.parametrize("layout", [NHD, HND])
@pytest.mark.parametrize("value,io", [("bf16", None), ("f16", None), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_types_and_layouts(value, io, layout, dim):
    check_attend(LENS, value=value, io=io, layout=layout, dim=dim)


@pytest.mark.parametrize("bs", [1, 3, 8, 20, 64, 200])
def test_attend_block_sizes(bs):
    check_attend(LENS, bs=bs, dim=128, layout=bs % 2)


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 9, 16, 17, 24, 40])
def test_attend_head_groups(group, value):
    check_attend([0, 5, 130, 40], group=group, value=value, hps=3, dim=128)


@pytest.mark.parametrize("value,dim", [("bf16", 8), ("bf16", 16), ("f16", 24), ("bf16", 72), ("bf16", 80), ("f16", 96), ("bf16", 160),
                                       ("f16", 192), ("bf16", 256), ("e4m3", 16), ("e4m3", 48), ("e4m3", 80), ("e4m3", 112),
                                       ("e4m3", 144), ("e4m3", 192), ("e4m3", 240), ("e4m3", 256)])
def test_attend_head_dims(value, dim):
    check_attend([70, 0, 1, 33], value=value, dim=dim, group=5)


@pytest.mark.parametrize("shards,hps", [(4, 2), (2, 1), (8, 1), (3, 2)])
def test_attend_shards(shards, hps):
    check_attend([300, 17, 64], shards=shards, hps=hps, dim=128, value="f16")


@pytest.mark.parametrize("window", [1, 7, 16, 100, 4000])
@pytest.mark.parametrize("bs", [16, 20])
def test_attend_window(window, bs):
    check_attend(LENS + [3000], window=window, dim=128, bs=bs)


@pytest.mark.parametrize("n_reqs,n", [(1, 8192), (1, 50000), (2, 20011), (17, 1500)])
@pytest.mark.parametrize("value", ["bf16", "e4m3"])
def test_attend_long(n_reqs, n, value):
    """Few long requests: the length is split over the GPU and joined."""
    check_attend([n + i for i in range(n_reqs)], dim=64, value=value, hps=1, group=3)


def test_attend_many_requests():
    rng = np.random.default_rng(5)
    check_attend(rng.integers(0, 40, 1500).tolist(), dim=64, hps=1, group=2)


@pytest.mark.parametrize("value,io", [("bf16", None), ("f16", None), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("group,dim,v_dim", [(16, 576, 512), (1, 576, 512), (37, 576, 512), (128, 576, 512), (8, 320, 256),
                                             (16, 64, 32), (16, 512, 512)])
def test_attend_latent(value, io, group, dim, v_dim):
    check_attend([0, 1, 63, 64, 65, 500, 1300], value=value, io=io, planes=1, hps=1, group=group, dim=dim, v_dim=v_dim, bs=64)


@pytest.mark.parametrize("bs,layout,hps", [(1, NHD, 1), (16, HND, 1), (20, NHD, 2), (128, HND, 2)])
def test_attend_latent_blocks_and_heads(bs, layout, hps):
    check_attend([3, 700, 0, 129], value="e4m3", planes=1, hps=hps, group=16, dim=576, v_dim=512, bs=bs, layout=layout, window=600)


@pytest.mark.parametrize("lens", [[1], [127, 128, 129], [640, 0, 64, 300], [5] * 40])
@pytest.mark.parametrize("bs", [4, 32, 64, 128, 256])
def test_attend_latent_runs_of_pages(bs, lens):
    """8-bit latents come in runs of the positions that a page holds in a row; a sequence's ends row by row."""
    check_attend(lens, value="e4m3", planes=1, hps=1, group=16, dim=576, v_dim=512, bs=bs)
    check_attend(lens, value="e4m3", planes=1, hps=1, group=16, dim=576, v_dim=512, bs=bs, window=100)


@pytest.mark.parametrize("shards,hps,dim,v_dim", [(2, 1, 576, 512), (1, 2, 512, 512), (1, 3, 144, 48)])
def test_attend_latent_shards_and_heads(shards, hps, dim, v_dim):
    check_attend([3, 700, 0, 129], value="e4m3", planes=1, shards=shards, hps=hps, group=5, dim=dim, v_dim=v_dim, bs=16)


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
def test_attend_latent_sharp_scores(value):
    """Maxima that move in many tiles, far apart, and queries of very different sizes."""
    case = Attend([2000, 300, 1], value=value, planes=1, hps=1, group=16, dim=576, v_dim=512, spread=4.0, scale=0.5)
    case.q *= torch.logspace(-3, 1, 16)[None, :, None]
    case.q = case.q.to(case.iodtype)
    case.check(*case.run())


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
def test_attend_latent_long(value):
    check_attend([30000, 1, 9000], value=value, planes=1, hps=1, group=16, dim=576, v_dim=512, bs=64)


@pytest.mark.parametrize("value", ["bf16", "f16"])
@pytest.mark.parametrize("lens", [[1], [63, 64, 65, 128], [640, 0, 64, 300], [5] * 40])
@pytest.mark.parametrize("bs", [1, 4, 20, 32, 64, 128])
def test_attend_latent_16_bit_runs_of_pages(value, lens, bs):
    check_attend(lens, value=value, planes=1, hps=1, group=16, dim=576, v_dim=512, bs=bs)
    check_attend(lens, value=value, planes=1, hps=1, group=16, dim=576, v_dim=512, bs=bs, window=100)


@pytest.mark.parametrize("shards,hps,dim,v_dim,layout", [(2, 1, 576, 512, NHD), (1, 2, 512, 512, NHD), (1, 2, 576, 512, NHD),
                                                         (1, 3, 144, 48, HND), (1, 1, 72, 8, NHD)])
@pytest.mark.parametrize("group", [5, 21])
def test_attend_latent_16_bit_shards_and_heads(shards, hps, dim, v_dim, layout, group):
    """Both kernels of 16-bit latents: the tensor maps cannot describe several shards, or heads with a gap."""
    check_attend([3, 700, 0, 129], value="bf16", planes=1, shards=shards, hps=hps, group=group, dim=dim, v_dim=v_dim, bs=16, layout=layout)


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("group", [17, 24, 32, 33, 48, 65])
def test_attend_latent_head_sets(value, group):
    """32 query heads at a time, in halves of 16: requests that one CTA answers, and long ones that several join."""
    check_attend([3000, 0, 1, 129, 20000], value=value, planes=1, hps=1, group=group, dim=576, v_dim=512, bs=64)
    check_attend([90] * 200, value=value, planes=1, hps=1, group=group, dim=576, v_dim=512, bs=16)


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
def test_attend_latent_head_sets_sharp_scores(value):
    case = Attend([2000, 300, 1], value=value, planes=1, hps=1, group=32, dim=576, v_dim=512, spread=4.0, scale=0.5)
    case.q *= torch.logspace(-3, 1, 32)[None, :, None]
    case.q = case.q.to(case.iodtype)
    case.check(*case.run())


@pytest.mark.parametrize("planes", [1, 2])
def test_attend_sharp_scores(planes):
    """Scores far apart: weights of one token, of none, and sums whose maximum moves late."""
    check_attend([400, 33, 1], planes=planes, hps=1, group=8, dim=64, v_dim=32 if planes == 1 else 0, spread=30.0, scale=1.0)


def test_attend_keeps_nan_and_infinity_of_live_positions():
    case = Attend([20, 20, 20], dim=64, hps=1, group=2)
    row = case.table[0, 0] * 16 + 3
    v = case.bufs[1].view(torch.bfloat16).view(-1, 64)
    v[row, 5] = float("nan")
    v[case.table[1, 0] * 16 + 4, 6] = float("inf")
    out, lse = case.run()
    assert torch.isnan(out[0, :, 5]).all() and torch.isfinite(out[0, :, :5]).all() and torch.isfinite(out[0, :, 6:]).all()
    assert not torch.isfinite(out[1, :, 6]).any() and torch.isfinite(out[1, :, :6]).all()
    assert torch.isfinite(out[2]).all() and torch.isfinite(lse).all()
    k = case.bufs[0].view(torch.bfloat16).view(-1, 64)
    k[row] = float("nan")
    out, lse = case.run()
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and torch.isfinite(lse[1:]).all()


@pytest.mark.parametrize("planes", [1, 2])
def test_attend_leaves_out_what_is_out_of_bounds(planes):
    case = Attend([100, 48, 30, 64], planes=planes, dim=64, hps=1, group=3, v_dim=64)
    table = case.table
    table[0, 2], table[1, 0], table[2, 0], table[2, 1] = -1, case.geom.n_blocks, 2 ** 31 - 1, -2 ** 31
    case.check(*case.run())
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_ERANGE
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    case.lens = [100, -3, 30, case.width * 16 + 1]
    out, lse = case.run()
    assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_ERANGE


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
def test_attend_latent_many_requests(value):
    rng = np.random.default_rng(6)
    check_attend(rng.integers(0, 90, 700).tolist(), value=value, planes=1, hps=1, group=3, dim=576, v_dim=512, bs=16)


def pinned(bufs):
    """The buffers again in pinned host memory, and the tensors that own it."""
    return [b.cpu().pin_memory() for b in bufs]


def test_pool_in_pinned_host_memory():
    case = Attend([100, 3], dim=64, hps=2, group=2)
    want = case.run()
    host = pinned(case.bufs)
    x = torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16)
    out = torch.zeros((2, 4 * 64), dtype=torch.bfloat16, device="cuda")
    with kvx.kvx_cache_create(kvx.Pool(case.geom, host), kvx.KVX_BF16, n_q_heads=4) as c:
        kvx.kvx_cache_attend(c, 0, case.d_q, 256, case.d_table, case.table.shape[1], case.width, case.d_len, 2, out, 256)
        slot = int(case.table[1, 0]) * 16 + 5
        kvx.kvx_cache_append(c, 0, x, 128, x, 128, dev(np.array([slot, -1], np.int64)), 2)
        assert kvx.kvx_cache_status(c) == kvx.KVX_OK
    assert torch.equal(out.view(2, 4, 64), want[0])
    assert all(torch.equal(b.view(torch.bfloat16).view(-1, 2, 64)[slot], x[0].cpu()) for b in host)


def test_latents_in_pinned_host_memory_are_refused():
    case = Attend([100, 3], planes=1, dim=64, hps=1, group=2, v_dim=64)
    case.run()
    with kvx.kvx_cache_create(kvx.Pool(case.geom, pinned(case.bufs)), kvx.KVX_BF16, n_q_heads=2) as c:
        with pytest.raises(kvx.KvxError) as ei:
            kvx.kvx_cache_attend(c, 0, case.d_q, 128, case.d_table, case.table.shape[1], case.width, case.d_len, 2, case.d_q, 128)
        assert ei.value.status == kvx.KVX_EUNSUPPORTED


@pytest.mark.parametrize("planes", [1, 2])
def test_attend_strides_streams_and_repeats(planes):
    case = Attend([700, 0, 90, 3000], planes=planes, dim=128, v_dim=128, hps=1, group=8)
    out, lse = case.run(pad=24)
    case.check(out, lse)
    stream = torch.cuda.Stream()
    for _ in range(3):
        again, lse2 = case.run(stream=stream)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert torch.equal(case.run(lse=False)[0], out) and (case.d_lse == 7.0).all()


def test_first_call_is_refused_in_a_capture_and_later_ones_replay():
    case = Attend([700, 5], dim=64, hps=2, group=2)
    want = case.run()
    fresh = Attend([700, 5], dim=64, hps=2, group=2)
    out = torch.zeros((2, 4 * 64), dtype=torch.bfloat16, device="cuda")
    fresh.d_q, fresh.d_table, fresh.d_len = case.d_q, case.d_table, case.d_len
    x = torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16)
    slots = dev(np.array([-1, -1], np.int64))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()

    def step(c):
        kvx.kvx_cache_append(c, 0, x, 128, x, 128, slots, 2, side)
        kvx.kvx_cache_attend(c, 0, case.d_q, 256, case.d_table, case.table.shape[1], case.width, case.d_len, 2, out, 256, None, side)

    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(kvx.KvxError) as ei:
            step(fresh.cache)
        assert ei.value.status == kvx.KVX_EINVAL and "capture" in str(ei.value)
        step(case.cache)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(2, 4, 64), want[0])


def test_attend_beyond_4_gib():
    """Blocks past 2^32 bytes of a buffer, and past 2^31 elements."""
    geom = PoolGeom(1, 2, 1, 8, 128, 2, 16, 140000)                        # 4.6 GB per plane
    bufs = [torch.zeros(geom.buffer_bytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    small = Attend([200], dim=128, hps=8, group=1, extra_blocks=0)
    far = np.full(small.table.shape, 2 ** 30, np.int32)
    far[0, :13] = 139999 - np.arange(13)
    for b, s in zip(bufs, small.bufs):
        size = 16 * 8 * 128 * 2
        for j in range(13):
            b[int(far[0, j]) * size:][:size] = s[int(small.table[0, j]) * size:][:size]
    want = small.run()
    with kvx.kvx_cache_create(kvx.Pool(geom, bufs), kvx.KVX_BF16) as c:
        out = torch.zeros((1, 8 * 128), dtype=torch.bfloat16, device="cuda")
        kvx.kvx_cache_attend(c, 0, small.d_q, 1024, dev(far), far.shape[1], 13, small.d_len, 1, out, 1024)
        torch.cuda.synchronize()
        assert torch.equal(out.view(1, 8, 128), want[0])
        x = torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16)
        kvx.kvx_cache_append(c, 0, x, 1024, x, 1024, dev(np.array([139999 * 16 + 15, 0], np.int64)), 2)
        assert kvx.kvx_cache_status(c) == kvx.KVX_OK
        for b in bufs:
            b = b.view(torch.bfloat16).view(-1, 8, 128)
            assert torch.equal(b[139999 * 16 + 15], x[0]) and torch.equal(b[0], x[1])
