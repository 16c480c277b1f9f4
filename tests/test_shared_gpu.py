"""GPU parity of kvx_cache_attend_shared against the plain 64-bit statement of attention (tests/decode_reference.py), within the
bounds of its arithmetic: every request over all its positions, as if nothing were shared."""
import numpy as np
import pytest

import decode_reference as ref
from shared_case import Shared, check_shared
from test_decode_gpu import HND, NHD, TYPES, dev, kvx, torch, typed

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


FORMS = [("bf16", None), ("f16", None), ("e4m3", "bf16"), ("e4m3", "f16")]


@pytest.mark.parametrize("value,io", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("prefix", [128, 300, 1000])
def test_one_group(value, io, dim, prefix):
    check_shared([(prefix, [1, 17, 40])], value=value, io=io, dim=dim)


def launches(case, **kw):
    before = kvx.kvx_launch_count()
    got = case.shared(**kw)
    return got, kvx.kvx_launch_count() - before


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
@pytest.mark.parametrize("bs", [1, 3, 8, 16, 20, 64, 200])
@pytest.mark.parametrize("layout", [NHD, HND])
def test_block_sizes_and_layouts(value, bs, layout):
    """Prefixes that end in a page, at its end and in a copy of it; groups, requests alone and empty ones in one batch."""
    check_shared([(128, [0, 1, 60]), 0, (257, [5, 0]), 90, (400, [129, 3, 3, 300])], value=value, bs=bs, layout=layout, dim=128, hps=2, group=4)


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 12, 16, 17, 24])
def test_head_groups(value, group):
    check_shared([(300, [9, 0, 70]), (140, [1, 1])], value=value, group=group, hps=3, dim=64)


@pytest.mark.parametrize("value,dim", [("bf16", 8), ("bf16", 16), ("f16", 24), ("bf16", 72), ("bf16", 80), ("f16", 96), ("bf16", 120),
                                       ("e4m3", 16), ("e4m3", 48), ("e4m3", 80), ("e4m3", 112)])
def test_head_dims(value, dim):
    check_shared([(500, [9, 0, 70]), (140, [1, 1])], value=value, group=5, dim=dim)


@pytest.mark.parametrize("shards,hps", [(4, 2), (2, 1), (8, 1), (3, 2)])
@pytest.mark.parametrize("value", ["f16", "e4m3"])
def test_shards(shards, hps, value):
    check_shared([(300, [9, 0, 70]), (140, [1, 1])], value=value, shards=shards, hps=hps, dim=128)


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("members,group,prefix", [(16, 8, 200), (17, 8, 200), (31, 4, 640), (32, 8, 1200), (33, 8, 130), (70, 8, 300),
                                                  (130, 1, 500), (300, 2, 129), (64, 16, 384)])
def test_rows(value, members, group, prefix):
    """128 rows of a slot, 256 of a unit: one slot in part filled, two, units of several row tiles."""
    check_shared([(prefix, [i % 7 for i in range(members)])], value=value, group=group, hps=1 if members > 60 else 2, dim=64 if members > 200 else 128)


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("prefix", [128, 129, 255, 256, 257, 383, 385, 5000, 20011])
@pytest.mark.parametrize("members", [2, 20])
def test_prefix_lengths(value, prefix, members):
    check_shared([(prefix, [3] * members)], value=value, group=8, hps=1, dim=128)


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
def test_long_prefix_of_two(value):
    """Few units: every CTA has a part of the same one."""
    check_shared([(40000, [100, 0])], value=value, group=1, hps=1, dim=64)


@pytest.mark.parametrize("n", [31, 32, 33, 63, 64, 65, 200, 1100])
def test_many_groups(n):
    """Beside the requests' own positions or before them, more than the plan takes at a time, and many units for a CTA."""
    rng = np.random.default_rng(n)
    check_shared([(int(rng.integers(100, 300)), rng.integers(0, 20, int(rng.integers(0, 4))).tolist()) for _ in range(n)],
                 group=2, hps=1 if n > 100 else 3, dim=64)


@pytest.mark.parametrize("value,io", FORMS)
@pytest.mark.parametrize("dim,group,rest", [(64, 8, [9000, 0, 700]), (128, 17, [3, 12000]), (80, 3, [40000, 1]), (128, 40, [2500] * 3), (64, 1, [70000, 300])])
def test_own_positions_of_several_ctas(value, io, dim, group, rest):
    """A few parts of a request's own positions, and more than are joined at a time."""
    check_shared([(300, rest), 5000], value=value, io=io, dim=dim, group=group, hps=1)


@pytest.mark.parametrize("value,io", FORMS)
@pytest.mark.parametrize("dim,layout,group,window", [(64, NHD, 2, 0), (128, HND, 3, 0), (80, NHD, 1, 250), (128, NHD, 17, 0)])
def test_many_requests(value, io, dim, layout, group, window):
    """Of every type, with groups of their own, a sliding window, and requests alone and empty."""
    rng = np.random.default_rng(7)
    groups = [(int(rng.integers(100, 400)), rng.integers(0, 90, 16).tolist()) for _ in range(20)] + [0, 70]
    check_shared(groups, value=value, io=io, dim=dim, layout=layout, group=group, hps=2, window=window)


@pytest.mark.parametrize("value,io", FORMS)
@pytest.mark.parametrize("dim,layout,group,window", [(64, NHD, 2, 0), (128, HND, 3, 0), (80, NHD, 1, 250), (128, NHD, 17, 0)])
def test_more_requests_than_are_planned_beside_the_rest(value, io, dim, layout, group, window):
    """The plan is a launch of its own."""
    rng = np.random.default_rng(8)
    groups = [(int(rng.integers(100, 400)), rng.integers(0, 60, 16).tolist()) for _ in range(25)] + [0, 70]
    case = Shared(groups, value=value, io=io, dim=dim, layout=layout, group=group, hps=1, window=window)
    got, n = launches(case)
    assert n == 4
    case.check_parts(*got)


@pytest.mark.parametrize("members,n_launches", [(383, 3), (384, 3), (385, 4)])
def test_where_the_plan_becomes_a_launch(members, n_launches):
    case = Shared([(200, [i % 9 for i in range(members)])], group=2, hps=1, dim=64)
    got, n = launches(case)
    assert n == n_launches
    case.check_parts(*got)


@pytest.mark.parametrize("n_groups,n_launches", [(256, 3), (257, 3), (384, 3), (385, 4), (2000, 4)])
def test_groups_without_members(n_groups, n_launches):
    """In front, between and behind those that have some."""
    case = Shared([(300, [1, 2]), 90, (200, [0, 5, 3])], dim=64)
    third = n_groups // 3
    off = [0] * third + [0, 2, 3] + [3] * (n_groups - 2 * third - 3) + [6] * (third + 1)
    prefix = [7] * third + [300, 90] + [150] * (n_groups - 2 * third - 3) + [200] + [9] * third
    assert len(off) == n_groups + 1 and len(prefix) == n_groups
    got, n = launches(case, off=off, prefix=prefix)
    assert n == n_launches
    case.check_parts(*got)
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK


@pytest.mark.parametrize("group,hps", [(130, 1), (256, 1), (300, 1), (140, 2)])
def test_more_than_128_query_heads_to_a_kv_head(group, hps):
    """Rows of one member in several units."""
    check_shared([(200, [40, 0, 300]), 150, 0], group=group, hps=hps, dim=64)


@pytest.mark.parametrize("members,group,hps", [(16, 8, 8), (32, 8, 8), (64, 8, 2), (9, 1, 152), (9, 1, 100), (20, 16, 3), (40, 8, 19)])
def test_one_group_whose_units_are_alike(members, group, hps):
    """As many CTAs for each unit, or not, where that would leave too many of them out."""
    check_shared([(2000, [i % 5 for i in range(members)])], group=group, hps=hps, dim=64)


def test_the_tensor_kernel_takes_what_is_worth_it():
    case = Shared([(300, [1, 2])], dim=64)
    assert launches(case)[1] > 1
    assert launches(case, max_blocks=case.width)[1] == 1                    # little to read twice
    wide = Shared([(300, [1, 2])], dim=192)
    assert kvx.kvx_cache_shared_bytes(wide.cache, 2, 1) == 0
    (out, lse), n = launches(wide)
    assert n == 1
    wide.check(out, lse)
    latent = Shared([(300, [1, 2])], planes=1, hps=1, dim=576, v_dim=512, value="e4m3", bs=64, group=16)
    latent.check(*latent.shared())
    for case in (Shared([300]), Shared([(300, [4])]), Shared([300, 20])):
        case.check_parts(*case.shared())
    none = Shared([(300, [1, 2])], dim=64)
    none.check_parts(*none.shared(off=[0], prefix=[]))


@pytest.mark.parametrize("say", [300, 301, 320, 359, 2 ** 31 - 1])
def test_a_prefix_beyond_the_shortest_member_is_cut_there(say):
    """What two members hold in the same blocks may be shared up to the shorter one's length."""
    case = Shared([(300, [0, 59])], say=[say], dim=64)
    case.check_parts(*case.shared())
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK


def test_less_of_the_prefix_may_be_named():
    case = Shared([(700, [0, 59, 3])], dim=64)
    for say in (0, 1, 127, 128, 300, 699):
        case.check_parts(*case.shared(prefix=[say]))


@pytest.mark.parametrize("window", [1, 100, 300, 359, 360, 4000])
def test_windows(window):
    """Shared while every member's window reaches the first position, read by each otherwise."""
    case = check_shared([(300, [0, 60]), (200, [1, 1]), 500], window=window, dim=128)
    case.check_parts(*case.shared())


def test_groups_that_are_no_list():
    """Reported, and then nothing is shared: the results are the same."""
    case = Shared([(300, [0, 60]), (200, [1, 1]), 50], dim=64)
    case.shared()
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    for off in ([0, 3, 2, 5], [-1, 2, 4, 5], [0, 2, 4, 6], [2, 0, 4, 5], [0, 2 ** 31 - 1, 4, 5], [0, -2 ** 31, 4, 5]):
        case.check_parts(*case.shared(off=off))
        assert kvx.kvx_cache_status(case.cache) == kvx.KVX_ERANGE
    case.check_parts(*case.shared(prefix=[300, -5, 50]))
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_ERANGE
    case.check_parts(*case.shared(off=[1, 1, 2], prefix=[50, 50]))          # requests before and behind the groups
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK


def test_blocks_and_lengths_out_of_bounds():
    case = Shared([(300, [0, 60]), (200, [1, 1]), 50], dim=64)
    case.table[:2, 3], case.table[2:4, 0], case.table[2:4, 1] = -1, case.geom.n_blocks, -2 ** 31
    case.check_parts(*case.shared())
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_ERANGE
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    case.table[:2, :300 // 16] = -1                                         # a prefix with nothing left but its end
    case.check_parts(*case.shared())
    kvx.kvx_cache_status(case.cache)
    lens = list(case.lens)
    lens[1] = -4                                                            # an empty member: nothing is shared with it
    out, lse = case.shared(lens=lens)
    assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_ERANGE
    case.lens = lens
    case.check_parts(out, lse)


def test_all_blocks_of_a_prefix_out_of_bounds():
    case = Shared([(256, [0, 0, 5])], dim=64, group=8)
    case.table[:, :16] = -1
    out, lse = case.shared()
    assert (out[:2] == 0).all() and (lse[:2] == -float("inf")).all()
    case.check_parts(out, lse)


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
def test_sharp_scores(value):
    """Scores far apart: weights of one position, of none, and maxima that move late."""
    case = Shared([(900, [0, 60]), (200, [1] * 20)], value=value, dim=64, spread=4.0, scale=0.5, group=8, hps=1)
    case.q = (case.q.float() * torch.logspace(-3, 1, 8)[None, :, None]).to(case.iodtype)
    case.check_parts(*case.shared())


@pytest.mark.parametrize("power", [114, -80])
@pytest.mark.parametrize("value", ["bf16", "e4m3"])
def test_queries_of_any_size(power, value):
    got = []
    for p in (0, power):
        case = Shared([(300, [1, 77])], value=value, dim=128, group=4, scale=2.0 ** -4 * 2.0 ** -p, seed=9)
        case.q = (case.q.double() * 2.0 ** p).to(case.iodtype)
        got.append(case.shared())
    assert torch.isfinite(got[0][0]).all() and torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def slots_of(case, r, at):
    return case.table[r, at // case.bs].astype(np.int64) * case.bs + at % case.bs


def plane(case, p):
    """The values of a plane of a token-major pool of one head and shard, [row][dim]."""
    return case.bufs[p].view({"bf16": torch.bfloat16, "f16": torch.float16}[case.value]).view(-1, case.dim)


@pytest.mark.parametrize("value", ["bf16", "f16"])
@pytest.mark.parametrize("members", [3, 40])
def test_nan_and_infinity(value, members):
    """An infinite value among the prefix' gives that infinity in that element alone, two of opposite sign and a NaN give NaN, to every
    member; a NaN key makes the members NaN, a NaN query its row; the other group keeps its bits."""
    case = Shared([(700, [5] * members), (300, [4, 4])], value=value, dim=64, hps=1, group=4)
    want, lse = case.shared()
    v = plane(case, 1)
    rng = np.random.default_rng(1)
    for d in range(0, 64, 2):
        v[int(slots_of(case, 0, rng.integers(0, 690))), d] = float("inf") if d % 4 else -float("inf")
    v[int(slots_of(case, 0, 3)), 1], v[int(slots_of(case, 0, 600)), 1] = float("inf"), -float("inf")
    v[int(slots_of(case, 0, 77)), 3] = float("nan")
    out, got = case.shared()
    assert torch.equal(got, lse)
    d = torch.arange(0, 64, 2, device="cuda")
    m = members
    assert (out[:m, :, d] == torch.where(d % 4 == 2, float("inf"), -float("inf"))).all()
    assert torch.isnan(out[:m, :, [1, 3]]).all()
    assert torch.equal(out[:m, :, 5::2], want[:m, :, 5::2]) and torch.equal(out[m:], want[m:])
    plane(case, 0)[int(slots_of(case, 0, 400)), 9] = float("nan")
    out, got = case.shared()
    assert torch.isnan(out[:m]).all() and torch.isnan(got[:m]).all() and torch.equal(out[m:], want[m:]) and torch.equal(got[m:], lse[m:])
    other = Shared([(700, [5] * members), (300, [4, 4])], value=value, dim=64, hps=1, group=4)
    other.q[1, 2, 7] = float("nan")
    other.q[2, 1, 7] = float("inf")
    out, got = other.shared()
    bad = torch.isnan(got)
    assert bad[1, 2] and bad.sum() <= 2 and torch.isnan(out[1, 2]).all()
    keep = torch.ones_like(bad)
    keep[1, 2] = keep[2, 1] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(got[keep], lse[keep])


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("gap", [14, 18, 24])
def test_weights_far_below_the_largest(value, gap):
    """A first position of large score and no value: the output is that of the thousands of small weights beside it."""
    rng = np.random.default_rng(11)
    size = 1000.0 if value == "f16" else 1.0
    both = Shared([(8193, [0, 0])], value=value, hps=1, group=4, dim=64, bs=64, seed=5, k_scale=0.25, v_scale=0.05)
    k, v = ref.one_large_score(rng, 8193, 1, 64, gap, 64 ** -0.5, 8.0, size)
    rows = ref.rows_of(both.table[0], np.arange(8193), 64, both.geom.n_blocks)
    put(both, rows, k, v)
    both.q[..., 0] = 8.0
    both.check_parts(*both.shared())


def put(case, rows, k, v):
    """Keys and values [n][1][dim] into the rows of the first member's table, and what the others have copied."""
    dtype = TYPES[case.value][1]
    for p, x in enumerate((k, v)):
        scale = (0.25, 0.05)[p] if case.value == "e4m3" else 1.0
        x = torch.from_numpy(x).float()
        x = (x / scale).clamp(-448, 448).to(dtype) if case.value == "e4m3" else x.to(dtype)
        raw = typed(case.bufs[p], case.geom, dtype).view(torch.uint8 if case.value == "e4m3" else torch.int16)
        n, bs = len(rows), case.bs
        raw[torch.from_numpy(rows // bs).cuda(), torch.from_numpy(rows % bs).cuda()] = x.contiguous().view(raw.dtype).cuda()
        case.host[p][rows] = x.double().numpy() * scale
        tail = n % bs
        for r in range(1, len(case.lens)):
            dst, src = int(case.table[r, n // bs]), int(case.table[0, n // bs])
            raw[dst, :tail] = raw[src, :tail]
            case.host[p][dst * bs:dst * bs + tail] = case.host[p][src * bs:src * bs + tail]


@pytest.mark.parametrize("value", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("spread", [0.3, 0.02])
def test_weights_of_nearly_equal_scores(value, spread):
    """Outputs that are small differences of large sums: a weight's rounding shows beside the output's."""
    case = Shared([(130, [0, 0])], value=value, hps=1, group=4, dim=64, bs=64, seed=5, k_scale=0.25, v_scale=0.05)
    k, v = ref.paired_values(np.random.default_rng(11), 130, 1, 64, spread)
    put(case, ref.rows_of(case.table[0], np.arange(130), 64, case.geom.n_blocks), k, v)
    case.check_parts(*case.shared())


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
def test_strides_streams_and_repeats(value):
    case = Shared([(700, [0, 90, 3]), 40, (3000, [5] * 20)], value=value, dim=128, hps=1, group=8)
    out, lse = case.shared(pad=24)
    case.check_parts(out, lse)
    stream = torch.cuda.Stream()
    for _ in range(3):
        again, lse2 = case.shared(stream=stream)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert torch.equal(case.shared(lse=False)[0], out) and (case.d_lse == 7.0).all()


def call(case, out, lse, space, stream, cache=None):
    n, hq = len(case.lens), case.heads * case.group
    kvx.kvx_cache_attend_shared(cache or case.cache, 0, case.d_q, hq * case.dim, case.d_table, case.d_table.shape[1], case.d_table.shape[1],
                                case.d_len, n, case.d_off, case.d_prefix, len(case.prefix), out, hq * case.dim, lse, space, space.numel(), stream)


def test_captured_and_replayed_with_other_lengths_and_groups():
    case = Shared([(700, [0, 90, 3]), 40, (300, [5] * 20)], dim=64, group=4)
    case.shared()
    n, hq = len(case.lens), case.heads * case.group
    out = torch.zeros((n, hq, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((n, hq), dtype=torch.float32, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call(case, out, lse, case.space, side)
    lens = np.array(case.lens)
    for cut, off in ((0, case.off), (30, case.off), (200, [0, 2, 3, 24]), (650, [0, 0, 0, 0])):
        now = np.maximum(lens - cut, 0)
        case.d_len.copy_(dev(now.astype(np.int32)))
        case.d_off.copy_(dev(np.asarray(off, np.int32)))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        keep, case.lens = case.lens, now.tolist()
        case.check_parts(out, lse)
        case.lens = keep
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK


def test_two_handles_on_two_streams():
    """Handles and workspaces of their own, on one pool, at the same time."""
    cases = [Shared([(3000, [9] * 20), 50], dim=128, group=8, hps=1, seed=s) for s in (1, 2)]
    want = [c.shared() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(w[0]) for w in want]
    lses = [torch.zeros_like(w[1]) for w in want]
    for c in cases:
        c.shared()
    for _ in range(20):
        for c, o, l, s in zip(cases, outs, lses, streams):
            call(c, o, l, c.space, s)
    torch.cuda.synchronize()
    for w, o, l in zip(want, outs, lses):
        assert torch.equal(w[0], o) and torch.equal(w[1], l)


def test_pool_in_pinned_host_memory():
    case = Shared([(300, [0, 60])], dim=64)
    want = case.shared()
    host = [b.cpu().pin_memory() for b in case.bufs]
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    with kvx.kvx_cache_create(kvx.Pool(case.geom, host), kvx.KVX_BF16, n_q_heads=case.heads * case.group) as c:
        call(case, out, lse, case.space, None, c)
        assert kvx.kvx_cache_status(c) == kvx.KVX_OK
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_buffers_past_4_gib():
    """The prefix' blocks at the end of buffers of 4.6 GB."""
    small = Shared([(300, [0, 60, 9])], dim=128, hps=8, group=1, extra_blocks=0)
    want = small.shared()
    geom = small.geom.replace(n_blocks=140000)
    bufs = [torch.zeros(geom.buffer_bytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    size = 16 * 8 * 128 * 2
    shift = 140000 - small.geom.n_blocks
    for b, s in zip(bufs, small.bufs):
        b[shift * size:] = s
    held = small.d_table < small.geom.n_blocks
    small.d_table = torch.where(held, small.d_table + shift, small.d_table)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    with kvx.kvx_cache_create(kvx.Pool(geom, bufs), kvx.KVX_BF16) as c:
        call(small, out, lse, small.space, None, c)
        assert kvx.kvx_cache_status(c) == kvx.KVX_OK
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("value", ["bf16", "e4m3"])
@pytest.mark.parametrize("groups", [[(3000, [9] * 3), 50, (200, [1, 1])], [(900, [2] * 40)], [(128, [0, 0])]])
@pytest.mark.parametrize("part", [1, 2, 3])
def test_a_wait_that_runs_out_is_reported(part, groups, value):
    """One part of the first CTA waits for what never comes: nothing faults, and the next call is right."""
    case = Shared(groups, value=value, dim=128, group=8, hps=1)
    out, lse = case.shared()
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    kvx.kvx_cache_inject_shared_stall(case.cache, part)
    case.shared()
    with pytest.raises(kvx.KvxError) as ei:
        kvx.kvx_cache_status(case.cache)
    assert ei.value.status == kvx.KVX_ETIMEDOUT
    again, lse2 = case.shared()
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    assert torch.equal(out, again) and torch.equal(lse, lse2)
