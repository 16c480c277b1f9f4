"""Operators of a decode worker whose requests share pages, as measured cases: the attention of a batch that shares
prefixes, the norm and rotation of new queries and keys on their way into the cache, and the forking, freeing and
compacting of a cache's pages.

`run` computes a case in its plain form (elementary torch operations in 32 bits) where `own` is false and by the
library's calls where it is true. `exact` states the same results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16, F16, E4M3 = "bf16", "f16", "e4m3"
DTYPE = {BF16: torch.bfloat16, F16: torch.float16, E4M3: torch.float8_e4m3fn}
SIZE = {BF16: 2, F16: 2, E4M3: 1}
NHD, HND = 0, 1
HALVES, PAIRS = 0, 1                                  # element i turns with i + dim / 2, or 2i with 2i + 1
PLAIN, LINEAR, BANDS, YARN = 0, 1, 2, 3               # how the frequencies are scaled for long contexts
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def shared_case(groups, members, prefix, rest, q_heads, heads, dim, shards=1, block=16, layout=NHD, value=BF16, io=BF16):
    """prefix: range of the tokens that the members of a group share; rest: of those that each has of its own."""
    return {"op": "shared", "groups": groups, "members": members, "prefix_lo": prefix[0], "prefix_hi": prefix[1], "rest_lo": rest[0],
            "rest_hi": rest[1], "q_heads": q_heads, "heads": heads, "dim": dim, "planes": 2, "shards": shards, "block": block,
            "layout": layout, "value": value, "io": io}


def rotate_case(tokens, run, q_heads, heads, dim, far, begin=0, turned=0, rule=HALVES, scaling=PLAIN, q_norm=True, k_norm=True,
                norm_dim=0, planes=2, shards=1, block=16, layout=NHD, value=BF16, io=BF16, padded=0):
    """run: consecutive tokens of one request; far: the largest position; [begin, begin + turned) is the part of a head that
    turns; padded: tokens in a hundred that carry no slot (-1)."""
    return {"op": "rotate", "tokens": tokens, "run": run, "q_heads": q_heads, "heads": heads, "dim": dim, "far": far, "begin": begin,
            "turned": turned or dim, "rule": rule, "scaling": scaling, "q_norm": q_norm, "k_norm": k_norm, "norm_dim": norm_dim or dim,
            "planes": planes, "shards": shards, "block": block, "layout": layout, "value": value, "io": io, "padded": padded}


def pages_case(op, n_reqs, lens, block, layers=1, planes=2, heads=8, dim=128, value=BF16, children=0, shared=0, idle=0, spare=1.2):
    """children: rows of the forked table; shared: blocks at the head of every row that all rows hold; idle: requests in a
    hundred that hold nothing any more; spare: blocks of the pool for each one that is held."""
    return {"op": op, "n_reqs": n_reqs, "len_lo": lens[0], "len_hi": lens[1], "block": block, "layers": layers, "planes": planes,
            "heads": heads, "dim": dim, "shards": 1, "layout": NHD, "value": value, "children": children, "shared": shared,
            "idle": idle, "spare": spare}


def listed():
    cases = [
        # the tiny pool: four requests on one short prompt, where latency is all
        ("shared_tiny", shared_case(1, 4, (200, 200), (1, 60), 8, 2, 64)),
        # 16 samples of one prompt of 8192 tokens, some hundred tokens into their answers
        ("shared_samples_16", shared_case(1, 16, (8192, 8192), (1, 400), 64, 8, 128)),
        # 64 questions about one document of 32768 tokens
        ("shared_document_64", shared_case(1, 64, (32768, 32768), (20, 500), 64, 8, 128)),
        # twelve system prompts with eight requests each over an 8-bit head-major cache, six query heads to a KV head
        ("shared_prompts_96", shared_case(12, 8, (1500, 4200), (1, 900), 24, 4, 128, block=24, layout=HND, value=E4M3, io=F16)),
        # one decode step of 64 sessions over the latent pool: only the last 64 elements turn, the latent alone is normed
        ("rotate_latent_64", rotate_case(64, 1, 16, 1, 576, 33000, begin=512, turned=64, rule=PAIRS, scaling=YARN, q_norm=False,
                                         norm_dim=512, planes=1, block=64, value=E4M3)),
        # a batch of prompts, 8192 tokens in all, with norms for each head and a long context's frequencies
        ("rotate_prompt_8192", rotate_case(8192, 2731, 64, 8, 128, 131072, scaling=BANDS)),
        # two prompts sampled eight times each: the partial last pages are copied in every layer
        ("fork_samples_16", pages_case("fork", 2, (1000, 3000), 16, layers=16, children=16)),
        # a step of a beam search: 96 of 128 beams go on, some in several, in another order
        ("fork_beams_128", pages_case("fork", 128, (300, 4000), 24, layers=8, heads=2, children=128)),
        # the free list of a small server of 40 requests
        ("free_small_40", pages_case("free", 40, (100, 3000), 16, shared=20, idle=10)),
        # that of 1024 sessions on a shared system prompt, a third of them gone
        ("free_sessions_1024", pages_case("free", 1024, (1024, 16000), 64, shared=16, idle=33)),
        # a pool that has emptied: what is left goes to its front
        ("compact_small", pages_case("compact", 12, (200, 2000), 16, layers=4, heads=2, idle=25, spare=2.0)),
        # the same of a large pool of 8-bit latents
        ("compact_latents", pages_case("compact", 64, (2048, 32768), 64, layers=8, planes=1, heads=1, dim=576, value=E4M3, idle=20, spare=1.5)),
    ]
    return [dict(c, name=n) for n, c in cases]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("shared", "shared", "rotate", "rotate", "fork", "free", "compact"))
    if op == "shared":
        value = rng.choice((BF16, F16, E4M3))
        shards = rng.choice((1, 1, 2, 4))
        heads = shards * rng.choice((1, 2))
        groups = log_int(rng, 1, 20)
        members = log_int(rng, 1, max(1, 200 // groups))
        hi = log_int(rng, 16, min(20000, 300000 // groups))
        return shared_case(groups, members, (hi // rng.choice((1, 1, 3)), hi), (rng.choice((0, 1)), log_int(rng, 1, 1500)),
                           heads * rng.choice((1, 2, 4, 5, 7, 8, 12, 16)), heads, rng.choice((64, 128)), shards=shards,
                           block=rng.choice((8, 16, 20, 32, 64)), layout=rng.choice((NHD, HND)), value=value,
                           io=value if value != E4M3 else rng.choice((BF16, F16)))
    if op == "rotate":
        far, scaling = log_int(rng, 100, 1000000), rng.choice((PLAIN, LINEAR, BANDS, YARN))
        if rng.random() < 0.3:
            return rotate_case(log_int(rng, 1, 5000), log_int(rng, 1, 4096), rng.choice((8, 16, 24)), 1, 576, far, begin=512, turned=64,
                               rule=PAIRS, scaling=scaling, q_norm=False, norm_dim=512, planes=1, block=rng.choice((16, 64)),
                               value=rng.choice((BF16, E4M3)), padded=rng.choice((0, 3)))
        value = rng.choice((BF16, F16, E4M3))
        shards = rng.choice((1, 1, 2, 4))
        heads, dim = shards * rng.choice((1, 2, 3)), rng.choice((64, 128))
        norm = rng.random() < 0.6
        return rotate_case(log_int(rng, 1, 8192), log_int(rng, 1, 4096), heads * rng.choice((1, 4, 7)), heads, dim, far,
                           turned=rng.choice((dim, dim, dim // 2)), rule=rng.choice((HALVES, PAIRS)), scaling=scaling, q_norm=norm,
                           k_norm=norm, shards=shards, block=rng.choice((8, 16, 20, 64)), layout=rng.choice((NHD, HND)), value=value,
                           io=value if value != E4M3 else rng.choice((BF16, F16)), padded=rng.choice((0, 3)))
    block = rng.choice((8, 16, 24, 64))
    if op == "fork":
        hi = log_int(rng, 10, 8000)
        n = log_int(rng, 1, max(1, min(200, 100000 // hi)))
        return pages_case("fork", n, (rng.choice((0, hi // 2)), hi), block, layers=rng.choice((1, 3, 8)), heads=rng.choice((1, 2, 8)),
                          dim=rng.choice((64, 128)), value=rng.choice((BF16, E4M3)), children=log_int(rng, 1, 256))
    if op == "free":
        hi = log_int(rng, 10, 16000)
        n = log_int(rng, 1, max(1, min(1500, 8000000 // hi)))
        return pages_case("free", n, (0, hi), block, shared=rng.choice((0, 1, hi // block // 2)), idle=rng.choice((0, 10, 60)),
                          spare=rng.choice((1.0, 1.3, 3.0)))
    hi = log_int(rng, 10, 16000)
    n = log_int(rng, 1, max(1, min(100, 200000 // hi)))
    return pages_case("compact", n, (0, hi), block, layers=rng.choice((1, 2, 5)), heads=rng.choice((1, 2)), dim=rng.choice((64, 128)),
                      value=rng.choice((BF16, E4M3)), shared=rng.choice((0, 1)), idle=rng.choice((0, 10, 60)), spare=rng.choice((1.2, 3.0)))


def work(case):
    if case["op"] == "shared":
        dim, n = case["dim"], case["groups"] * case["members"]
        prefix, rest = (case["prefix_lo"] + case["prefix_hi"]) / 2, (case["rest_lo"] + case["rest_hi"]) / 2      # spread evenly
        per_token = 2 * case["heads"] * dim * SIZE[case["value"]] + 4 / case["block"]
        return {"bytes": (case["groups"] * prefix + n * rest) * per_token + n * (case["q_heads"] * (4 * dim + 4) + 4),
                "flops": n * (prefix + rest) * case["q_heads"] * 4 * dim}
    if case["op"] == "rotate":
        n, dim = case["tokens"], case["dim"]
        q, kv = n * case["q_heads"] * dim, n * case["planes"] * case["heads"] * dim
        return {"bytes": q * 4 + kv * (2 + SIZE[case["value"]]) + 12 * n, "flops": 8 * q + 6 * kv}
    mean = (case["len_lo"] + case["len_hi"]) / 2 * (1 - case["idle"] / 100)
    entries = case["n_reqs"] * (mean / case["block"] + 0.5)
    block_bytes = case["layers"] * case["planes"] * case["block"] * case["heads"] * case["dim"] * SIZE[case["value"]]
    if case["op"] == "fork":                            # the last page of a row is nearly always in part filled
        rows = case["children"]
        copies = max(1.0, rows - min(case["n_reqs"], 0.64 * rows))
        return {"bytes": rows * (mean / case["block"] * 8 + 16) + copies * (2 * block_bytes + 12), "flops": rows * mean / case["block"]}
    n_blocks = entries * case["spare"]
    if case["op"] == "free":
        return {"bytes": entries * 4 + n_blocks * 4 + (n_blocks - entries) * 4, "flops": entries + n_blocks}
    moves = entries * (1 - 1 / case["spare"])
    return {"bytes": n_blocks * 4 + entries * 8 + moves * (2 * block_bytes + 8), "flops": n_blocks}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def normal(shape, dtype, gen, scale=1.0):
    """N(0, 1) values in the tensor's type; 8-bit codes stand for value / scale."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        x = torch.randn(n, generator=gen, device="cuda")
        flat[i:i + n] = (x.div_(scale).clamp_(-E4M3_MAX, E4M3_MAX) if dtype == torch.float8_e4m3fn else x).to(dtype)
    return out


class Geometry:
    def __init__(self, **counts):
        self.__dict__.update(counts)


def buffers(case, n_blocks, gen, scale, layers=1):
    """One tensor per (layer, plane, shard), in the pool's own layout."""
    hps = case["heads"] // case["shards"]
    inner = (case["block"], hps) if case["layout"] == NHD else (hps, case["block"])
    return [normal((n_blocks, *inner, case["dim"]), DTYPE[case["value"]], gen, scale) for _ in range(layers * case["planes"] * case["shards"])]


def cache_of(case, n_blocks, bufs, scales, q_heads, layers=1):
    """The handle that a serving program keeps for its pool."""
    from disaggregated_prefill_decode_gb300 import kvx
    code = {BF16: kvx.KVX_BF16, F16: kvx.KVX_F16, E4M3: kvx.KVX_E4M3}
    geom = Geometry(n_layers=layers, n_planes=case["planes"], n_shards=case["shards"], heads_per_shard=case["heads"] // case["shards"],
                    head_dim=case["dim"], elem_bytes=SIZE[case["value"]], block_size=case["block"], layout=case["layout"], n_blocks=n_blocks)
    io = case.get("io") or (BF16 if case["value"] == E4M3 else case["value"])
    return kvx.kvx_cache_create(kvx.Pool(geom, bufs), value_type=code[case["value"]], io_type=code[io], n_q_heads=q_heads,
                                k_scale=scales[0], v_scale=scales[1])


def spread(rng, n, lo, hi, share_without=0):
    """n numbers spread evenly over [lo, hi], some of them 0, in an order of the seed's."""
    x = np.floor(lo + (hi - lo + 1) * (np.arange(n) + 0.5) / n).astype(np.int64)
    some = np.arange(n) * share_without // 100
    x[np.flatnonzero(np.diff(some, prepend=0))] = 0
    return rng.permutation(x).astype(np.int32)


def scales_of(case, rng):
    if case["value"] != E4M3:
        return 1.0, 1.0
    a, b = (float(np.float32(rng.uniform(0.012, 0.02))) for _ in range(2))
    return (a, b) if case["planes"] == 2 else (a, a)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case}
    {"shared": prepare_shared, "rotate": prepare_rotate}.get(case["op"], prepare_pages)(case, state, rng, gen)
    return state


def prepare_shared(case, state, rng, gen):
    groups, members, bs = case["groups"], case["members"], case["block"]
    n = groups * members
    prefix = spread(rng, groups, case["prefix_lo"], case["prefix_hi"])
    rest = spread(rng, n, case["rest_lo"], case["rest_hi"])
    lens = np.repeat(prefix, members) + rest
    held = -(-lens // bs)
    whole = prefix // bs                                # pages of the prefix that are full: one copy for the group
    n_ids = int(whole.sum() + (held - np.repeat(whole, members)).sum())
    n_blocks = int(1.2 * n_ids) + 8
    ids = rng.permutation(n_blocks).astype(np.int32)
    width = max(int(held.max()), 1)
    table = np.full((n, width), -1, np.int32)
    at, tails = 0, []
    for g in range(groups):
        shared = ids[at:at + whole[g]]
        at += whole[g]
        for r in range(g * members, (g + 1) * members):
            table[r, :whole[g]] = shared
            table[r, whole[g]:held[r]] = ids[at:at + held[r] - whole[g]]
            at += held[r] - whole[g]
            if prefix[g] % bs:                          # a page that the prefix ends in: each member's begins with a copy of it
                tails.append((table[g * members, whole[g]], table[r, whole[g]], prefix[g] % bs))
    scales = scales_of(case, rng)
    bufs = buffers(case, n_blocks, gen, scales[0])
    for b in bufs:
        raw = b.view(torch.uint8)
        for src, dst, m in tails:
            if src != dst:
                part = (slice(0, int(m)),) if case["layout"] == NHD else (slice(None), slice(0, int(m)))
                raw[(int(dst), *part)] = raw[(int(src), *part)]
    q, d = case["q_heads"], case["dim"]
    state.update(bufs=bufs, scales=scales, lens=dev(lens.astype(np.int32)), table=dev(table), width=width, n=n,
                 prefix=dev(prefix), off=dev((np.arange(groups + 1) * members).astype(np.int32)),
                 longest=int(prefix.max()), most=int(rest.max()),
                 q=normal((n, q, d), DTYPE[case["io"]], gen), out=torch.zeros((n, q, d), dtype=DTYPE[case["io"]], device="cuda"),
                 lse=torch.zeros((n, q), dtype=torch.float32, device="cuda"))
    if own:
        from disaggregated_prefill_decode_gb300 import kvx
        state["cache"] = cache_of(case, n_blocks, bufs, scales, q)
        size = kvx.kvx_cache_shared_bytes(state["cache"], n, groups)
        state["space"] = torch.empty(size, dtype=torch.uint8, device="cuda")


def frequencies(case):
    """Of the pairs of the part that turns, in radians a position, and the factor of what has turned."""
    d = case["turned"]
    f = 10000.0 ** (-2 * np.arange(d // 2, dtype=np.float64) / d) if case["scaling"] != BANDS else 500000.0 ** (-2 * np.arange(d // 2, dtype=np.float64) / d)
    s = 8.0
    if case["scaling"] == LINEAR:
        return f / s, 1.0
    if case["scaling"] == BANDS:                        # long waves are stretched, short ones kept, those between blended
        t = np.clip((8192 * f / (2 * np.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f / s * (1 - t) + f * t, 1.0
    if case["scaling"] == YARN:
        turn = lambda b: d * math.log(4096 / (2 * math.pi * b)) / (2 * math.log(10000.0))
        lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), d - 1)
        r = np.clip((np.arange(d // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / s * r + f * (1 - r), 0.1 * math.log(s) + 1.0
    return f, 1.0


def rotation_of(case):
    from disaggregated_prefill_decode_gb300 import kvx
    code = {PLAIN: kvx.KVX_ROTATE_PLAIN, LINEAR: kvx.KVX_ROTATE_LINEAR, BANDS: kvx.KVX_ROTATE_BANDS, YARN: kvx.KVX_ROTATE_YARN}
    more = {BANDS: dict(base=500000.0, factor=8.0, low=1.0, high=4.0, original=8192.0), LINEAR: dict(factor=8.0),
            YARN: dict(factor=8.0, low=1.0, high=32.0, original=4096.0), PLAIN: {}}[case["scaling"]]
    return kvx.kvx_rotation_create(layout=kvx.KVX_ROTATE_PAIRS if case["rule"] == PAIRS else kvx.KVX_ROTATE_HALVES, begin=case["begin"],
                                   dim=case["turned"], scaling=code[case["scaling"]], norm_dim=case["norm_dim"], eps=1e-6, **more)


def prepare_rotate(case, state, rng, gen):
    n, bs, dim = case["tokens"], case["block"], case["dim"]
    left, runs = n, []
    while left:                                         # tokens of one request after another
        runs.append(min(left, case["run"]))
        left -= runs[-1]
    first = rng.integers(0, max(1, case["far"] - case["run"]), len(runs))
    need = [-(-(f % bs + r) // bs) for f, r in zip(first.tolist(), runs)]
    n_blocks = int(1.2 * sum(-(-(bs - 1 + r) // bs) for r in runs)) + 8
    order = rng.permutation(n_blocks)
    at, slots, positions = 0, [], []
    for f, r, k in zip(first.tolist(), runs, need):
        t = f % bs + np.arange(r)
        slots.append(order[at:at + k][t // bs].astype(np.int64) * bs + t % bs)
        positions.append(f + np.arange(r))
        at += k
    slots = np.concatenate(slots)
    slots[rng.random(n) < case["padded"] / 100] = -1
    scales = scales_of(case, rng)
    bufs = buffers(case, n_blocks, gen, scales[0])
    q, kv, io = case["q_heads"] * dim, case["heads"] * dim, DTYPE[case["io"]]
    stride = q + case["planes"] * kv                    # one projection gives queries, keys and values side by side
    x = normal((n, stride), io, gen)
    freq, factor = frequencies(case)
    state.update(bufs=bufs, scales=scales, slots=dev(slots), positions=dev(np.concatenate(positions).astype(np.int32)), stride=stride,
                 x=x, q=x[:, :q].view(n, case["q_heads"], dim), k=x[:, q:q + kv].view(n, case["heads"], dim),
                 v=x[:, q + kv:].view(n, case["heads"], dim) if case["planes"] == 2 else None,
                 q_weight=(normal((case["norm_dim"],), torch.float32, gen) * 0.2 + 1).to(io) if case["q_norm"] else None,
                 k_weight=(normal((case["norm_dim"],), torch.float32, gen) * 0.2 + 1).to(io) if case["k_norm"] else None,
                 freq=dev(freq), factor=factor, out=torch.zeros((n, case["q_heads"], dim), dtype=io, device="cuda"))
    if own:
        state["cache"] = cache_of(case, n_blocks, bufs, scales, case["q_heads"])
        state["rotation"] = rotation_of(case)


def prepare_pages(case, state, rng, gen):
    n, bs, op = case["n_reqs"], case["block"], case["op"]
    lens = spread(rng, n, case["len_lo"], case["len_hi"], case["idle"])
    held = -(-lens // bs)
    shared = np.minimum(held, case["shared"])
    n_ids = int(shared.max() + (held - shared).sum())
    n_blocks = int(case["spare"] * n_ids) + (case["children"] if op == "fork" else 1)
    ids = rng.permutation(n_blocks).astype(np.int32)
    head = ids[:shared.max()]
    width = max(int(held.max()), 1)
    table = np.full((n, width), -1, np.int32)
    at = int(shared.max())
    for r in range(n):
        table[r, :shared[r]] = head[:shared[r]]
        table[r, shared[r]:held[r]] = ids[at:at + held[r] - shared[r]]
        at += held[r] - shared[r]
    refs = np.bincount(table[table >= 0], minlength=n_blocks).astype(np.int32)
    result = torch.zeros(3, dtype=torch.int64, device="cuda")
    state.update(n_blocks=n_blocks, table=dev(table), width=width, lens=dev(lens), result=result)
    if op == "free":
        state.update(refs=torch.zeros(n_blocks, dtype=torch.int32, device="cuda"), left=int((refs == 0).sum()),
                     free=torch.zeros(n_blocks, dtype=torch.int32, device="cuda"))
        return
    bufs = buffers(case, n_blocks, gen, 1.0, case["layers"])
    state["bufs"] = bufs
    if op == "fork":
        rows = case["children"]
        survivors = rng.permutation(n)[:max(1, n * 3 // 4)] if rows <= n else np.arange(n)
        parent = survivors[rng.integers(0, len(survivors), rows)].astype(np.int32)
        # the first row that goes on from a request keeps its last page, the others get copies
        seen, copies = set(), 0
        for p in parent.tolist():
            copies += bool(lens[p] % bs) and p in seen
            seen.add(p)
        state.update(parent=dev(parent), spare_ids=dev(ids[at:]), copies=copies,
                     new_table=torch.zeros((rows, width), dtype=torch.int32, device="cuda"),
                     new_lens=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                     src=torch.zeros(rows, dtype=torch.int32, device="cuda"), dst=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                     scratch=torch.zeros(n, dtype=torch.int32, device="cuda"))
    else:
        live = int((refs > 0).sum())
        moves = int((refs[live:] > 0).sum())
        most = n_blocks // 2 + 1
        state.update(refs=dev(refs), live=live, moves=moves, most=most, new_table=torch.zeros((n, width), dtype=torch.int32, device="cuda"),
                     src=torch.zeros(most, dtype=torch.int32, device="cuda"), dst=torch.zeros(most, dtype=torch.int32, device="cuda"))
    if own:
        state["cache"] = cache_of(case, n_blocks, bufs, (1.0, 1.0), case["heads"], case["layers"])


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"shared": own_shared, "rotate": own_rotate, "fork": own_fork, "free": own_free, "compact": own_compact}[op](state)
    return {"shared": plain_shared, "rotate": plain_rotate, "fork": plain_fork, "free": plain_free, "compact": plain_compact}[op](state)


def own_shared(s):
    from disaggregated_prefill_decode_gb300 import kvx
    c = s["case"]
    kvx.kvx_cache_attend_shared(s["cache"], 0, s["q"], c["q_heads"] * c["dim"], s["table"], s["width"], s["width"], s["lens"], s["n"],
                                s["off"], s["prefix"], c["groups"], s["out"], c["q_heads"] * c["dim"], s["lse"], s["space"], s["space"].numel())
    return s["out"], s["lse"]


def own_rotate(s):
    from disaggregated_prefill_decode_gb300 import kvx
    c = s["case"]
    kvx.kvx_cache_append_rotated(s["cache"], 0, s["rotation"], s["q"], s["stride"], s["q_weight"], s["out"], c["q_heads"] * c["dim"],
                                 s["k"], s["stride"], s["k_weight"], s["v"], s["stride"], s["positions"], s["slots"], c["tokens"])
    return [s["out"], *s["bufs"]]


def own_fork(s):
    from disaggregated_prefill_decode_gb300 import kvx
    c = s["case"]
    kvx.kvx_pages_fork(s["table"], s["width"], s["width"], s["lens"], c["n_reqs"], s["parent"], c["children"], c["block"],
                       s["spare_ids"], s["spare_ids"].numel(), s["new_table"], s["width"], s["new_lens"], s["src"], s["dst"],
                       s["scratch"], s["result"])
    kvx.kvx_cache_copy(s["cache"], 0, c["layers"], s["src"], s["dst"], c["children"])
    return [s["new_table"], s["new_lens"], s["src"], s["dst"], s["result"], *s["bufs"]]


def own_free(s):
    from disaggregated_prefill_decode_gb300 import kvx
    c = s["case"]
    kvx.kvx_pages_free(s["table"], s["width"], s["width"], s["lens"], c["n_reqs"], c["block"], s["n_blocks"], s["refs"], s["free"], s["result"])
    return s["refs"], s["free"], s["result"]


def own_compact(s):
    from disaggregated_prefill_decode_gb300 import kvx
    c = s["case"]
    kvx.kvx_pages_compact(s["table"], s["width"], s["width"], s["lens"], c["n_reqs"], c["block"], s["refs"], s["n_blocks"],
                          s["new_table"], s["width"], s["src"], s["dst"], s["most"], s["result"])
    kvx.kvx_cache_copy(s["cache"], 0, c["layers"], s["src"], s["dst"], s["most"])
    return [s["new_table"], s["src"], s["dst"], s["result"], *s["bufs"]]


def gathered(s, plane, table):
    """[row][position][head][dim] of the blocks of a table, from every shard, in 32 bits."""
    c = s["case"]
    parts = []
    for i in range(c["shards"]):
        x = s["bufs"][plane * c["shards"] + i][table].float()
        x = x.transpose(2, 3) if c["layout"] == HND else x
        parts.append(x.reshape(x.shape[0], -1, *x.shape[3:]))
    return torch.cat(parts, 2) if len(parts) > 1 else parts[0]


def plain_shared(s):
    """The prefix of a group is gathered and multiplied once for all its members, the rest request by request."""
    c = s["case"]
    groups, members, heads, dim, bs = c["groups"], c["members"], c["heads"], c["dim"], c["block"]
    n, each = s["n"], c["q_heads"] // c["heads"]
    q = s["q"].float().view(n, heads, each, dim) * (s["scales"][0] / math.sqrt(dim))
    table = s["table"].long().clamp(min=0)
    first = table[::members, :-(-s["longest"] // bs)]
    own_cols = s["prefix"].repeat_interleave(members, output_size=n).long()[:, None] // bs + torch.arange(-(-s["most"] // bs) + 1, device="cuda")
    own_table = table.gather(1, own_cols.clamp(max=s["width"] - 1))
    k0, v0 = gathered(s, 0, first), gathered(s, 1, first)
    k1, v1 = gathered(s, 0, own_table), gathered(s, 1, own_table)
    # [group][head][member, query] x positions of the prefix, then each request's own positions
    q0 = q.view(groups, members, heads, each, dim).transpose(1, 2).reshape(groups, heads, members * each, dim)
    s0 = torch.matmul(q0, k0.permute(0, 2, 3, 1))
    s0 = s0.masked_fill((torch.arange(k0.shape[1], device="cuda") >= s["prefix"][:, None])[:, None, None], float("-inf"))
    s1 = torch.matmul(q, k1.permute(0, 2, 3, 1))
    start = s["prefix"].repeat_interleave(members, output_size=n)
    pos = start[:, None] // bs * bs + torch.arange(k1.shape[1], device="cuda")
    s1 = s1.masked_fill(((pos < start[:, None]) | (pos >= s["lens"][:, None]))[:, None, None], float("-inf"))
    top0 = s0.amax(3).reshape(groups, heads, members, each).transpose(1, 2).reshape(n, heads, each, 1)
    top = torch.maximum(top0, s1.amax(3, keepdim=True))
    top = torch.where(top == float("-inf"), 0.0, top)
    p0 = torch.exp(s0 - top.reshape(groups, members, heads, each).transpose(1, 2).reshape(groups, heads, members * each, 1))
    p1 = torch.exp(s1 - top)
    back = lambda x: x.reshape(groups, heads, members, each, -1).transpose(1, 2).reshape(n, heads, each, -1)
    total = back(p0.sum(3)) + p1.sum(3, keepdim=True)
    out = back(torch.matmul(p0, v0.permute(0, 2, 1, 3))) + torch.matmul(p1, v1.permute(0, 2, 1, 3))
    s["out"].copy_((out * s["scales"][1] / torch.where(total == 0, 1.0, total)).reshape(n, heads * each, dim))
    s["lse"].copy_((top + torch.log(total)).reshape(n, heads * each))
    return s["out"], s["lse"]


def normed(x, weight, n, eps=1e-6):
    if weight is None:
        return x
    y = x[..., :n] * torch.rsqrt(x[..., :n].square().mean(-1, keepdim=True) + eps) * weight.float()
    return y if n == x.shape[-1] else torch.cat([y, x[..., n:]], -1)


def turned(s, x):
    c = s["case"]
    lo, d = c["begin"], c["turned"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    part = x[..., lo:lo + d]
    if c["rule"] == HALVES:
        a, b = part[..., :d // 2], part[..., d // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x[..., :lo], y, x[..., lo + d:]], -1)


def plain_rotate(s):
    c = s["case"]
    hps = c["heads"] // c["shards"]
    q = turned(s, normed(s["q"].float(), s["q_weight"], c["norm_dim"]))
    k = turned(s, normed(s["k"].float(), s["k_weight"], c["norm_dim"]))
    keep = s["slots"] >= 0
    s["out"].copy_(torch.where(keep[:, None, None], q.to(s["out"].dtype), s["out"]))
    blk, at = (s["slots"] // c["block"])[keep], (s["slots"] % c["block"])[keep]
    for p, x in enumerate((k, s["v"])[:c["planes"]]):
        x = x[keep].float()
        if c["value"] == E4M3:
            x = (x * float(np.float32(1.0) / np.float32(s["scales"][p]))).clamp(-E4M3_MAX, E4M3_MAX)
        x = x.to(DTYPE[c["value"]])
        for i in range(c["shards"]):
            buf, part = s["bufs"][p * c["shards"] + i], x[:, i * hps:(i + 1) * hps]
            buf, part = (buf.view(torch.uint8), part.contiguous().view(torch.uint8)) if c["value"] == E4M3 else (buf, part)
            if c["layout"] == NHD:
                buf[blk, at] = part
            else:
                buf[blk, :, at] = part
    return [s["out"], *s["bufs"]]


def copied(s, src, dst):
    for b in s["bufs"]:
        raw = b.view(torch.uint8)
        raw[dst] = raw[src]


def plain_fork(s):
    c = s["case"]
    rows, bs = c["children"], c["block"]
    parent, row = s["parent"].long(), torch.arange(rows, device="cuda")
    lens = s["lens"][parent]
    held = (lens.long() + bs - 1) // bs
    first = torch.full((c["n_reqs"],), rows, device="cuda").scatter_reduce(0, parent, row, "amin")[parent]
    need = (lens % bs != 0) & (first != row)
    k = torch.cumsum(need, 0) - need.long()
    table = s["table"][parent]
    last = (held - 1).clamp(min=0)[:, None]
    mine = table.gather(1, last)[:, 0]
    to = torch.where(need, s["spare_ids"][torch.where(need, k, 0)], mine)
    table = table.scatter(1, last, to[:, None])
    s["new_table"].copy_(torch.where(torch.arange(s["width"], device="cuda") < held[:, None], table, -1))
    s["new_lens"].copy_(lens)
    at = torch.where(need, k, rows)
    for name, x in (("src", mine), ("dst", to)):
        s[name].copy_(torch.full((rows + 1,), -1, dtype=torch.int32, device="cuda").scatter_(0, at, x)[:rows])
    s["result"][0] = held.sum()
    s["result"][1] = need.sum()
    s["result"][2] = 0
    if s["copies"]:
        copied(s, s["src"][:s["copies"]].long(), s["dst"][:s["copies"]].long())
    return [s["new_table"], s["new_lens"], s["src"], s["dst"], s["result"], *s["bufs"]]


def plain_free(s):
    c, n = s["case"], s["n_blocks"]
    held = (s["lens"].long() + c["block"] - 1) // c["block"]
    live = torch.arange(s["width"], device="cuda") < held[:, None]
    refs = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    refs.scatter_add_(0, torch.where(live, s["table"], n).view(-1).long(), torch.ones(live.numel(), dtype=torch.int32, device="cuda"))
    s["refs"].copy_(refs[:n])
    order = torch.argsort((s["refs"] > 0).int(), stable=True)
    s["free"][:s["left"]] = order[:s["left"]].int()
    s["result"][0] = (s["refs"] > 0).sum()
    s["result"][1] = n - s["result"][0]
    s["result"][2] = 0
    return s["refs"], s["free"], s["result"]


def plain_compact(s):
    c, n = s["case"], s["n_blocks"]
    live = s["refs"] > 0
    front = torch.arange(n, device="cuda") < live.sum()
    moves = s["moves"]
    src = torch.argsort((~(live & ~front)).int(), stable=True)[:moves]        # held, behind the front
    dst = torch.argsort((~(~live & front)).int(), stable=True)[:moves]        # free, in the front
    to = torch.arange(n, dtype=torch.int32, device="cuda")
    to[src] = dst.int()
    held = (s["lens"].long() + c["block"] - 1) // c["block"]
    mine = torch.arange(s["width"], device="cuda") < held[:, None]
    s["new_table"].copy_(torch.where(mine, to[s["table"].long().clamp(min=0)], s["table"]))
    for name, x in (("src", src), ("dst", dst)):
        s[name].fill_(-1)
        s[name][:moves] = x.int()
    s["result"][0] = live.sum()
    s["result"][1] = moves
    s["result"][2] = 0
    if moves:
        copied(s, src, dst)
    return [s["new_table"], s["src"], s["dst"], s["result"], *s["bufs"]]


# ------------------------------------------------------------------------------------------------
# the same in 64 bits
# ------------------------------------------------------------------------------------------------

def exact(case, seed):
    """Attention: one request at a time over all its positions, softmax by its definition. Rotation: products with complex
    numbers of modulus 1, before any rounding. Pages are whole numbers and copies: None."""
    if case["op"] not in ("shared", "rotate"):
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return (exact_shared if case["op"] == "shared" else exact_rotate)(case, s)


def exact_shared(case, s):
    n, dim, bs, each = s["n"], case["dim"], case["block"], case["q_heads"] // case["heads"]
    out = torch.zeros((n, case["q_heads"], dim), dtype=torch.float64, device="cuda")
    lse = torch.full((n, case["q_heads"]), float("-inf"), dtype=torch.float64, device="cuda")
    hps = case["heads"] // case["shards"]
    for r, length in enumerate(s["lens"].tolist()):
        if not length:
            continue
        pos = torch.arange(length, device="cuda")
        blk, slot = s["table"][r, pos // bs].long(), pos % bs
        for h in range(case["heads"]):
            k, v = (s["bufs"][p * case["shards"] + h // hps] for p in (0, 1))
            pick = (blk, slot, h % hps) if case["layout"] == NHD else (blk, h % hps, slot)
            rows = slice(h * each, (h + 1) * each)
            scores = s["q"][r, rows].double() @ (k.view(torch.uint8)[pick].view(k.dtype).double() * s["scales"][0]).T / math.sqrt(dim)
            lse[r, rows] = torch.logsumexp(scores, 1)
            out[r, rows] = torch.softmax(scores, 1) @ (v.view(torch.uint8)[pick].view(v.dtype).double() * s["scales"][1])
    return out, lse


def exact_rotate(case, s):
    lo, d, m = case["begin"], case["turned"], case["norm_dim"]
    unit = torch.polar(torch.full_like(s["freq"], s["factor"])[None].expand(case["tokens"], -1).contiguous(),
                       s["positions"].double()[:, None] * s["freq"])[:, None]

    def both(x, weight):
        x = x.double().clone()
        if weight is not None:
            x[..., :m] = x[..., :m] / torch.sqrt((x[..., :m] ** 2).sum(-1, keepdim=True) / m + 1e-6) * weight.double()
        part = x[..., lo:lo + d]
        z = torch.complex(part[..., :d // 2], part[..., d // 2:]) if case["rule"] == HALVES else torch.view_as_complex(part.reshape(*part.shape[:-1], d // 2, 2).contiguous())
        z = torch.view_as_real(z * unit)
        x[..., lo:lo + d] = torch.cat([z[..., 0], z[..., 1]], -1) if case["rule"] == HALVES else z.flatten(-2)
        return x

    slots = s["slots"].cpu().numpy()
    rows = np.flatnonzero(slots >= 0)
    tok, blk, at = dev(rows), dev(slots[rows] // case["block"]), dev(slots[rows] % case["block"])
    out = torch.zeros((case["tokens"], case["q_heads"], case["dim"]), dtype=torch.float64, device="cuda")
    out[tok] = both(s["q"], s["q_weight"])[tok]
    outs = [out]
    hps = case["heads"] // case["shards"]
    for p in range(case["planes"]):
        x = (both(s["k"], s["k_weight"]) if p == 0 else s["v"].double())[tok] / s["scales"][p]
        x = torch.clamp(x, -E4M3_MAX, E4M3_MAX) if case["value"] == E4M3 else x
        for i in range(case["shards"]):
            buf = s["bufs"][p * case["shards"] + i].double()
            for h in range(hps):
                if case["layout"] == NHD:
                    buf[blk, at, h] = x[:, i * hps + h]
                else:
                    buf[blk, h, at] = x[:, i * hps + h]
            outs.append(buf)
    return outs
