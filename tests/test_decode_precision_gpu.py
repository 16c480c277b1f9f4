"""Precision of the attention's weights: inputs on which a weight's rounding, or the loss of small weights, shows beside the
output's own rounding, against the 64-bit statement within the bounds of weights held in parts (tests/decode_reference.py)."""
import numpy as np
import pytest

import decode_reference as ref
from test_decode_gpu import HND, NHD, TYPES, Attend, kvx, torch, typed

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


class Filled(Attend):
    """An Attend whose keys and values come from fill(n) -> (keys, values), [n][heads][dim]; of latents the values are the
    first v_dim elements, the keys those after them, and the queries see the keys alone."""

    def __init__(self, lens, fill, q0=0.0, **kw):
        super().__init__(lens, **kw)
        scales = (kw.get("k_scale", 0.03), kw.get("v_scale", 0.05) if len(self.host) == 2 else kw.get("k_scale", 0.03))
        vt, vdtype, esz = TYPES[self.value]
        for r, n in enumerate(lens):
            if not n:
                continue
            rows = ref.rows_of(self.table[r], np.arange(n), self.bs, self.geom.n_blocks)
            k, v = fill(n)
            planes = (k, v)
            if len(self.host) == 1:
                planes = (np.concatenate([v, k], 2),)
            for p, x in enumerate(planes):
                x = torch.from_numpy(x).float()
                scale = scales[p] if self.value == "e4m3" else 1.0
                x = (x / scale).clamp(-448, 448).to(vdtype) if self.value == "e4m3" else x.to(vdtype)
                self.host[p][rows] = x.double().numpy() * scale
                hps = self.geom.heads_per_shard
                for s in range(self.geom.n_shards):
                    view = typed(self.bufs[p * self.geom.n_shards + s], self.geom, vdtype)
                    raw = view.view(torch.uint8 if esz == 1 else torch.int16)
                    part = x[:, s * hps:(s + 1) * hps].contiguous().view(raw.dtype).cuda()
                    raw[torch.from_numpy(rows // self.bs).cuda(), torch.from_numpy(rows % self.bs).cuda()] = part
        first = self.v_dim if len(self.host) == 1 else 0
        self.q[..., :first] = 0
        if q0:
            self.q[..., first] = q0

    def check_parts(self, out, lse, parts):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for r, n in enumerate(self.lens):
            rows = ref.rows_of(self.table[r], np.arange(n), self.bs, self.geom.n_blocks)
            for h in range(self.heads):
                hs = slice(h * self.group, (h + 1) * self.group)
                k, v = self.host[0][rows, h], self.host[-1][rows, h, :self.v_dim]
                o, l, weight, spread, floor = ref.attend(self.q[r, hs].double().numpy(), k, v, self.scale)
                if n == 0:
                    assert (out[r, hs] == 0).all() and (lse[r, hs] == -np.inf).all()
                    continue
                b_out, b_lse = ref.parts_bounds(o, l, weight, spread, floor, self.dim, n, self.io, parts)
                off = np.abs(out[r, hs] - o) / b_out
                assert (off <= 1).all(), (r, h, n, off.max())
                assert (np.abs(lse[r, hs] - l) <= b_lse).all(), (r, h, n)


# value, io, planes, shards, query heads a KV head, head_dim, v_dim, what a weight is held in
PLANES = [("bf16", None, 2, 1, 4, 64, 0, "bf16 planes"), ("bf16", None, 2, 2, 12, 128, 0, "bf16 planes"), ("f16", None, 2, 1, 4, 64, 0, "f16"),
          ("f16", None, 2, 1, 12, 128, 0, "f16"), ("f16", None, 2, 1, 2, 192, 0, "f16"), ("e4m3", "f16", 2, 1, 8, 128, 0, "f16"),
          ("e4m3", "bf16", 2, 1, 8, 128, 0, "f16"), ("e4m3", "bf16", 2, 1, 16, 64, 0, "f16"), ("e4m3", "bf16", 2, 1, 3, 256, 0, "f16")]
WARPS = [("bf16", None, 1, 2, 16, 576, 512, "bf16"), ("f16", None, 1, 2, 5, 576, 512, "f16"), ("e4m3", "f16", 1, 2, 16, 576, 512, "f16"),
         ("e4m3", "bf16", 1, 2, 16, 576, 512, "f16")]
TENSOR = [("bf16", None, 1, 1, 16, 576, 512, "bf16"), ("bf16", None, 1, 1, 32, 576, 512, "bf16"), ("f16", None, 1, 1, 16, 576, 512, "f16 tensor"),
          ("f16", None, 1, 1, 24, 576, 512, "f16 tensor")]
CODES = [("e4m3", "bf16", 1, 1, 16, 576, 512, "4 codes"), ("e4m3", "f16", 1, 1, 7, 576, 512, "4 codes"),
         ("e4m3", "bf16", 1, 1, 32, 576, 512, "4 codes, wide"), ("e4m3", "bf16", 1, 1, 70, 576, 512, "4 codes, wide"),
         ("e4m3", "f16", 1, 1, 40, 576, 512, "4 codes")]
CASES = PLANES + WARPS + TENSOR + CODES


def run(fill_of, lens, form, q0=0.0, **kw):
    value, io, planes, shards, group, dim, v_dim, parts = form
    rng = np.random.default_rng(11)
    width = dim - v_dim if planes == 1 else dim
    case = Filled(lens, lambda n: fill_of(rng, n, shards, dim, v_dim or dim, width, planes), q0=q0, value=value, io=io, planes=planes,
                  shards=shards, hps=1, group=group, dim=dim, v_dim=v_dim, bs=64, layout=HND if shards == 1 else NHD, seed=5, **kw)
    case.check_parts(*case.run(), parts)
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    kvx.kvx_cache_destroy(case.cache)


@pytest.mark.parametrize("spread", [0.3, 0.02, 0.002])
@pytest.mark.parametrize("form", CASES)
def test_weights_of_nearly_equal_scores(form, spread):
    def fill(rng, n, heads, dim, v_dim, width, planes):
        k, v = ref.paired_values(rng, n, heads, max(width, v_dim), spread)
        return k[..., :width], v[..., :v_dim]
    run(fill, [2, 3, 0, 6, 17, 40], form)


@pytest.mark.parametrize("gap", [14, 16, 18, 24])
@pytest.mark.parametrize("form", CASES)
def test_weights_far_below_the_largest(form, gap):
    """A first position of large score and no value: the output is that of the thousands of small weights beside it."""
    value, io, planes, shards, group, dim, v_dim, parts = form
    size = 1000.0 if "f16" in (value, io) else 1.0

    def fill(rng, n, heads, dim, v_dim, width, planes):
        k, v = ref.one_large_score(rng, n, heads, max(width, v_dim), gap, dim ** -0.5, 8.0, size if planes == 2 or value != "e4m3" else 1.0)
        return k[..., :width], v[..., :v_dim]
    run(fill, [8193, 700, 1], form, q0=8.0, k_scale=0.25, v_scale=0.05 * size)


def raw_values(case, plane):
    """The values of a plane of one shard and one head, [row][dim]."""
    return case.bufs[plane].view(TYPES[case.value][1]).view(-1, case.dim)


@pytest.mark.parametrize("value", ["bf16", "f16"])
@pytest.mark.parametrize("group,dim", [(1, 64), (8, 128), (12, 128), (3, 256)])
@pytest.mark.parametrize("lens,window", [([1, 40, 9000], 0), ([2, 600, 20011], 300)])
def test_an_infinite_value_gives_that_infinity(value, group, dim, lens, window):
    """sum p v with one infinite v is that infinity, in that element alone; with two of opposite sign it is NaN."""
    case = Attend(lens, value=value, dim=dim, hps=1, group=group, window=window, seed=2)
    before = case.run()
    v = raw_values(case, 1)
    rng = np.random.default_rng(1)
    for r, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        for d in range(0, dim, 2):                                         # every other element, a position of its own
            v[int(ref.rows_of(case.table[r], np.array([rng.integers(first, n)]), 16, case.geom.n_blocks)[0]), d] = (
                float("inf") if d % 4 else -float("inf"))
        at = [first, n - 1]
        rows = ref.rows_of(case.table[r], np.array(at), 16, case.geom.n_blocks)
        if n > 1:
            v[int(rows[0]), 1], v[int(rows[1]), 1] = float("inf"), -float("inf")
        if first:                                                          # before the window: no matter what
            rows = ref.rows_of(case.table[r], np.arange(first), 16, case.geom.n_blocks)
            v[torch.from_numpy(rows).cuda(), 3] = float("nan")
            v[torch.from_numpy(rows).cuda(), 5] = float("inf")
    out, lse = case.run()
    assert torch.equal(lse, before[1])
    d = torch.arange(0, dim, 2, device="cuda")
    assert (out[:, :, d] == torch.where(d % 4 == 2, float("inf"), -float("inf"))).all()
    assert torch.equal(out[:, :, 3::2], before[0][:, :, 3::2])
    assert torch.isnan(out[1:, :, 1]).all() and torch.equal(out[0, :, 1].isnan(), torch.full((group,), lens[0] > 1, device="cuda"))
    kvx.kvx_cache_destroy(case.cache)


@pytest.mark.parametrize("planes,shards,group,dim,v_dim", [(2, 1, 4, 128, 0), (2, 1, 12, 64, 0), (1, 1, 16, 576, 512), (1, 1, 24, 576, 512),
                                                           (1, 2, 8, 576, 512)])
@pytest.mark.parametrize("value", ["bf16", "e4m3"])
@pytest.mark.parametrize("power", [114, -80])
def test_queries_of_any_size(power, value, planes, shards, group, dim, v_dim):
    """Queries times a power of two and a scale that undoes it: the same bits."""
    got = []
    for p in (0, power):
        case = Attend([300, 1, 77], value=value, planes=planes, shards=shards, hps=1, group=group, dim=dim, v_dim=v_dim, bs=64,
                      scale=2.0 ** -4 * 2.0 ** -p, seed=9)
        case.q = (case.q.double() * 2.0 ** p).to(case.iodtype)
        got.append(case.run())
        kvx.kvx_cache_destroy(case.cache)
    assert torch.isfinite(got[0][0]).all() and torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("form", TENSOR + CODES + WARPS)
def test_queries_with_a_few_large_elements(form):
    """The others of the row are far below the largest, which is what 8-bit products bring them up by."""
    value, io, planes, shards, group, dim, v_dim, parts = form
    case = Attend([300, 1, 2000], value=value, io=io, planes=planes, shards=shards, hps=1, group=group, dim=dim, v_dim=v_dim, bs=64, seed=13)
    case.q = case.q.float()
    case.q[:, :, [5, 200, 570]] *= 300.0
    case.q = case.q.to(case.iodtype)
    case.check(*case.run())
    kvx.kvx_cache_destroy(case.cache)
