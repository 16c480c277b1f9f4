"""GPU parity of kvx_cache_append_rotated against a plain 64-bit statement (tests/rotate_reference.py), within the bounds of
32-bit arithmetic and one rounding."""
import numpy as np
import pytest

import kvx_inputs
import rotate_reference as ref

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


def f64(x):
    return x.double().cpu().numpy()


class Case:
    """A pool full of marks, tokens in a projection's rows, and the rotation."""

    def __init__(self, value="bf16", io=None, q_heads=4, heads=2, dim=64, planes=2, shards=1, block=16, layout=NHD, tokens=37, far=5000,
                 q_norm=True, k_norm=True, seed=0, size=1.0, scales=(0.0, 0.0), with_q=True, **rotation):
        self.io = io or ("bf16" if value == "e4m3" else value)
        self.value, self.q_heads, self.heads, self.dim, self.planes, self.tokens = value, q_heads, heads, dim, planes, tokens
        rng = np.random.default_rng(seed)
        self.geom = PoolGeom(2, planes, shards, heads // shards, dim, TYPES[value][2], block, tokens // block + 9, layout)
        self.bufs = [torch.full((self.geom.buffer_bytes,), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(self.geom.n_buffers)]
        self.slots = rng.permutation(self.geom.n_blocks * block)[:tokens].astype(np.int64)
        self.slots[rng.random(tokens) < 0.1] = -1
        self.pos = rng.integers(0, far, tokens).astype(np.int32)
        dtype = TYPES[self.io][1]
        self.row = (q_heads + planes * heads) * dim
        self.x = dev(rng.standard_normal((tokens, self.row)) * size).to(dtype)
        self.weights = [dev(1 + 0.3 * rng.standard_normal(rotation.get("norm_dim") or dim)).to(dtype) if on else None for on in (q_norm, k_norm)]
        self.rotation, self.scales, self.with_q = rotation, scales, with_q
        self.eps = rotation.get("eps") or 1e-6

    def slices(self, x):
        q, kv = self.q_heads * self.dim, self.heads * self.dim
        return x[:, :q], x[:, q:q + kv], x[:, q + kv:] if self.planes == 2 else None

    def run(self, in_place=False, stream=None, status=kvx.KVX_OK):
        q, k, v = self.slices(self.x)
        self.before = [f64(p) for p in self.slices(self.x) if p is not None]
        out = q if in_place else torch.full((self.tokens, self.q_heads * self.dim), 77.0, dtype=self.x.dtype, device="cuda")
        self.out_before = f64(out)
        with kvx.kvx_cache_create(kvx.Pool(self.geom, self.bufs), TYPES[self.value][0], io_type=TYPES[self.io][0], n_q_heads=self.q_heads,
                                  k_scale=self.scales[0], v_scale=self.scales[1] if self.planes == 2 else 0.0) as cache, \
                kvx.kvx_rotation_create(**self.rotation) as r:
            kvx.kvx_cache_append_rotated(cache, 1, r, q if self.with_q else None, self.row, self.weights[0], out if self.with_q else None,
                                         self.row if in_place else self.q_heads * self.dim, k, self.row, self.weights[1], v, self.row,
                                         dev(self.pos), dev(self.slots), self.tokens, stream)
            assert kvx.kvx_cache_status(cache, stream) == status
            self.freq, self.magnitude = kvx.kvx_rotation_get(r)
        return out

    def stated(self, x, weight, heads):
        w = None if weight is None else f64(weight)
        return ref.rotated(x.reshape(self.tokens, heads, self.dim), w, self.pos, self.freq, self.magnitude, self.rotation.get("begin", 0),
                           self.rotation.get("layout", 0) == 1, self.rotation.get("norm_dim") or self.dim, self.eps)

    def check(self, out):
        keep = (self.slots >= 0) & (self.slots < self.geom.n_blocks * self.geom.block_size)
        got = f64(out).reshape(self.tokens, self.q_heads, self.dim)
        if self.with_q:
            want, err = self.stated(self.before[0], self.weights[0], self.q_heads)
            off = np.abs(got - want) - ref.bound(want, err, self.io)
            assert (off[keep] <= 0).all(), off[keep].max()
            assert np.array_equal(got[~keep], self.out_before.reshape(got.shape)[~keep])
        else:
            assert (got == 77).all()
        g, hps, block = self.geom, self.geom.heads_per_shard, self.geom.block_size
        per = g.n_planes * g.n_shards
        for b in self.bufs[:per]:
            assert (b == 0x5a).all()                                          # the other layer
        for p in range(self.planes):
            x = self.before[1 + p].reshape(self.tokens, self.heads, self.dim)
            want, err = self.stated(x, self.weights[1], self.heads) if p == 0 else (x, np.zeros_like(x))
            scale = float(np.float32(self.scales[p if self.planes == 2 else 0] or 1.0))
            if self.value == "e4m3":
                want, err = ref.stored(want, err, scale)
            for s in range(g.n_shards):
                buf = self.bufs[per + p * g.n_shards + s]
                shape = (g.n_blocks, block, hps, self.dim) if g.layout == NHD else (g.n_blocks, hps, block, self.dim)
                rows = buf.view(TYPES[self.value][1]).view(shape)
                raw = buf.view(-1).cpu().numpy().reshape(*shape[:3], -1)
                touched = np.zeros(shape[:3], bool)
                for t in np.flatnonzero(keep):
                    blk, at = divmod(int(self.slots[t]), block)
                    touched[(blk, at) if g.layout == NHD else (blk, slice(None), at)] = True
                assert (raw[~touched] == 0x5a).all()                          # no other slot
                vals = f64(rows.float())
                for t in np.flatnonzero(keep):
                    blk, at = divmod(int(self.slots[t]), block)
                    have = vals[blk, at] if g.layout == NHD else vals[blk, :, at]
                    w, e = want[t, s * hps:(s + 1) * hps], err[t, s * hps:(s + 1) * hps]
                    if p == 1 and self.value != "e4m3":
                        assert np.array_equal(have, w)
                    else:
                        off = np.abs(have - w) - ref.bound(w, e, self.value)
                        assert (off <= 0).all(), off.max()


BANDS = dict(scaling=2, base=500000.0, factor=8.0, low=1.0, high=4.0, original=8192.0)
YARN = dict(scaling=3, factor=8.0, original=4096.0)


@pytest.mark.parametrize("value,io", [("bf16", None), ("f16", None), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("kw", [
    dict(dim=64), dict(dim=128, q_heads=8), dict(dim=256, q_heads=2), dict(dim=128, q_heads=14, heads=2, layout_=HND, shards=2),
    dict(dim=80, turned=32), dict(dim=80, turned=80), dict(dim=96, turned=48, begin=32), dict(dim=16, q_heads=6, heads=3, block=5),
    dict(dim=128, pairs=True), dict(dim=128, pairs=True, turned=64, begin=64), dict(dim=64, pairs=True, turned=24, begin=8),
    dict(dim=128, turned=0), dict(dim=128, q_norm=False, k_norm=False), dict(dim=64, q_norm=False), dict(dim=64, k_norm=False),
    dict(dim=128, norm_dim=64), dict(dim=128, with_q=False), dict(dim=240, turned=16, begin=224, norm_dim=232),
    dict(dim=64, tokens=1), dict(dim=128, tokens=3000, q_heads=7, heads=1, far=200000)])
def test_rotate(value, io, kw):
    kw = dict(kw, scales=(0.02, 0.013) if value == "e4m3" else (0.0, 0.0))
    turned, rotation = kw.pop("turned", kw["dim"]), dict(layout=int(kw.pop("pairs", False)))
    c = make(value, io, kw.pop("layout_", NHD), rotation, turned, kw)
    c.check(c.run())


def make(value, io, pool_layout, rotation, turned, kw):
    """A case whose pool has `pool_layout`; the rotation's own layout and part of the head are passed apart."""
    begin, norm_dim = kw.pop("begin", 0), kw.pop("norm_dim", 0)
    c = Case(value, io, layout=pool_layout, norm_dim=norm_dim, **kw)
    c.rotation = dict(dim=turned, begin=begin, norm_dim=norm_dim, **rotation)
    return c


@pytest.mark.parametrize("scaling", [dict(), dict(scaling=1, factor=4.0), BANDS, YARN, dict(YARN, magnitude=0.5)])
@pytest.mark.parametrize("pairs", [0, 1])
def test_far_positions(scaling, pairs):
    """Up to the last position that 32 bits hold: angles in 32 bits would be off by hundreds of turns."""
    for far in (10, 131072, 2 ** 20, 2 ** 24):
        c = make("f16", None, NHD, dict(layout=pairs, **scaling), 128, dict(dim=128, far=far, tokens=50, seed=far))
        c.pos[0], c.pos[1] = 0, far - 1
        c.check(c.run())


def test_negative_positions_turn_back():
    c = make("f16", None, NHD, dict(layout=0), 64, dict(dim=64))
    c.pos = -c.pos
    c.check(c.run())


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_heads", [1, 16, 24])
def test_latents(value, q_heads):
    """The last 64 elements of a latent turn, the first 512 are normed; queries are not normed."""
    c = make(value, None, NHD, dict(layout=1, **YARN), 64, dict(dim=576, q_heads=q_heads, heads=1, planes=1, block=64, tokens=130, far=40000,
                                                                 begin=512, norm_dim=512, q_norm=False, scales=(0.03, 0.0) if value == "e4m3" else (0, 0)))
    c.check(c.run())


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_norm,k_norm", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("pairs,begin,turned,norm_dim", [(1, 0, 64, 0), (0, 512, 64, 512), (1, 264, 48, 8), (1, 8, 256, 576), (0, 320, 256, 64), (1, 0, 0, 264)])
def test_parts_of_wide_heads(value, q_norm, k_norm, pairs, begin, turned, norm_dim):
    """Two slots of a head for each lane, some of which only copy."""
    for dim in (576, 520 if begin + turned <= 520 and norm_dim <= 520 and value == "bf16" else 576):
        c = make(value, None, NHD, dict(layout=pairs), turned, dict(dim=dim, q_heads=3, heads=1, planes=1, block=16, tokens=70, begin=begin, norm_dim=norm_dim,
                                                                    q_norm=q_norm, k_norm=k_norm, scales=(0.03, 0.0) if value == "e4m3" else (0, 0)))
        c.check(c.run())


@pytest.mark.parametrize("tokens", [2, 9, 76, 152, 305, 611, 1217, 2433])
@pytest.mark.parametrize("wide", [False, True])
def test_numbers_of_tokens(tokens, wide):
    """A token's heads among many warps, a few, or one."""
    kw = dict(dim=576, q_heads=8, heads=1, planes=1, begin=512, norm_dim=512, q_norm=False) if wide else dict(dim=64, q_heads=24, heads=2)
    c = make("bf16", None, NHD, dict(layout=int(wide)), 64, dict(kw, tokens=tokens))
    c.check(c.run())


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
def test_in_place(value):
    c = make(value, None, HND, dict(layout=0), 128, dict(dim=128, q_heads=8, heads=2, tokens=200))
    c.check(c.run(in_place=True))


def test_slots_outside_are_reported_and_skipped():
    c = make("bf16", None, NHD, dict(layout=0), 64, dict(dim=64, tokens=20))
    c.slots[[3, 7]] = (c.geom.n_blocks * 16, -2)
    c.check(c.run(status=kvx.KVX_ERANGE))


def test_small_rows_saturation_and_nan():
    """Rows of zeros and of tiny values (eps keeps them), values beyond the largest code, NaN in one head alone."""
    c = make("e4m3", "bf16", NHD, dict(layout=0, eps=1e-5), 64, dict(dim=64, tokens=30, scales=(0.001, 0.001)))
    c.eps = 1e-5
    c.x[0] = 0
    c.x[1] *= 1e-6
    c.x[2] *= 1e4
    c.slots[:3] = np.setdiff1d(np.arange(c.geom.n_blocks * 16), c.slots)[:3]
    c.check(c.run())
    d = make("bf16", None, NHD, dict(layout=0), 64, dict(dim=64, tokens=5, q_heads=4, heads=2, seed=1))
    d.slots = np.arange(5, dtype=np.int64)
    clean = d.run()
    d.bufs = [torch.full_like(b, 0x5a) for b in d.bufs]
    d.x[2, 64 + 5] = float("nan")                                              # query head 1 of token 2
    d.x[3, 4 * 64 + 7] = float("inf")                                          # key head 0 of token 3
    out = d.run()
    bad = torch.isnan(out.view(5, 4, 64)).any(2).cpu().numpy()
    assert bad.sum() == 1 and bad[2, 1]
    keep = ~bad
    assert torch.equal(out.view(5, 4, 64)[dev(keep)], clean.view(5, 4, 64)[dev(keep)])
    keys = d.bufs[2].view(torch.bfloat16).view(-1, 16, 2, 64)[0, :5]
    assert torch.isnan(keys).any(2).sum() == 1 and torch.isnan(keys[3, 0]).any()


def test_captured_and_replayed():
    """Captured on a side stream, replayed with other tokens, positions and slots."""
    c = make("bf16", None, NHD, dict(layout=0), 64, dict(dim=64, tokens=16))
    q, k, v = c.slices(c.x)
    out, pos, slots = torch.full((16, 256), 77.0, dtype=torch.bfloat16, device="cuda"), dev(c.pos), dev(c.slots)
    side = torch.cuda.Stream()
    with kvx.kvx_cache_create(kvx.Pool(c.geom, c.bufs), 1, n_q_heads=4) as cache, kvx.kvx_rotation_create(dim=64) as r:
        def call():
            kvx.kvx_cache_append_rotated(cache, 1, r, q, c.row, c.weights[0], out, 256, k, c.row, c.weights[1], v, c.row, pos, slots, 16, side)
        torch.cuda.synchronize()
        call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        kvx.kvx_rotation_destroy(r)                                            # the graph has the frequencies
        for seed in (3, 4):
            d = make("bf16", None, NHD, dict(layout=0), 64, dict(dim=64, tokens=16, seed=seed))
            c.x.copy_(d.x)
            pos.copy_(dev(d.pos))
            slots.copy_(dev(d.slots))
            out.fill_(77.0)
            for b in c.bufs:
                b.fill_(0x5a)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            c.pos, c.slots = d.pos, d.slots
            c.before, c.out_before = [f64(p) for p in c.slices(c.x)], np.full((16, 256), 77.0)
            c.freq, c.magnitude = np.array(ref.frequencies(64)), 1.0
            c.check(out)
