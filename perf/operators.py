"""The decode side's operators over a paged KV pool, as measured cases: slot maps built from request lengths,
the append of new keys and values, and the attention of one new token per request.

`run` computes a case in its plain form (elementary torch operations in 32 bits) where `own` is false and by the
library's calls where it is true. `exact` states the same results in 64 bits, one request at a time.
"""
import math

import numpy as np
import torch

own = False

BF16, F16, E4M3 = "bf16", "f16", "e4m3"
DTYPE = {BF16: torch.bfloat16, F16: torch.float16, E4M3: torch.float8_e4m3fn}
SIZE = {BF16: 2, F16: 2, E4M3: 1}
NHD, HND = 0, 1
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def slots_case(n_reqs, block, ctx, new, idle=0):
    """ctx, new: ranges of the cached and the new tokens of a request; idle: requests in a hundred without new tokens."""
    return {"op": "slots", "n_reqs": n_reqs, "block": block, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "idle": idle}


def append_case(tokens, run, heads, dim, planes=2, shards=1, block=16, layout=NHD, value=BF16, io=BF16, padded=0):
    """run: consecutive tokens of one request; padded: tokens in a hundred that carry no slot (-1)."""
    return {"op": "append", "tokens": tokens, "run": run, "heads": heads, "dim": dim, "planes": planes, "shards": shards,
            "block": block, "layout": layout, "value": value, "io": io, "padded": padded}


def attend_case(n_reqs, lens, q_heads, heads, dim, planes=2, v_dim=0, shards=1, block=16, layout=NHD, value=BF16, io=BF16,
                window=0, empty=0):
    """lens: range of the cached tokens; empty: requests in a hundred with none."""
    return {"op": "attend", "n_reqs": n_reqs, "len_lo": lens[0], "len_hi": lens[1], "q_heads": q_heads, "heads": heads,
            "dim": dim, "planes": planes, "v_dim": v_dim, "shards": shards, "block": block, "layout": layout,
            "value": value, "io": io, "window": window, "empty": empty}


def listed():
    cases = [
        # one decode step of the batched push's 16 requests: one new token each, a block now and then
        ("slots_decode_16", slots_case(16, 16, (1024, 8192), (1, 1))),
        # a mixed step of a busy server: decoding requests, chunks of prefill, requests that wait; an odd block size
        ("slots_mixed_777", slots_case(777, 24, (0, 4096), (1, 512), idle=30)),
        # 256 sessions of the multi-turn workload placed at once, latent blocks of 64 tokens
        ("slots_sessions_256", slots_case(256, 64, (0, 1024), (2048, 32768))),
        # the keys and values of one decode step, 16 requests, token-major
        ("append_decode_16", append_case(16, 1, 8, 128)),
        # one prompt of 8192 tokens written head-major into four head shards
        ("append_prompt_8192", append_case(8192, 8192, 8, 128, shards=4, layout=HND, value=F16, io=F16)),
        # a long prefill's latents quantised to 8 bits, with the padding of a fixed batch
        ("append_latent_50001", append_case(50001, 700, 1, 576, planes=1, block=64, value=E4M3, padded=2)),
        # the tiny pool: four short requests, where latency is all
        ("attend_tiny", attend_case(4, (100, 300), 8, 2, 64)),
        # one long request: the cache's length has to be split over the GPU
        ("attend_single_8192", attend_case(1, (8192, 8192), 64, 8, 128)),
        # the batched workload's requests, token-major
        ("attend_batched_16", attend_case(16, (1024, 8192), 64, 8, 128)),
        # four head shards of two heads, requests up to 16384 tokens, one of them alone many times another
        ("attend_shards_tp4", attend_case(8, (2048, 16384), 32, 8, 128, shards=4, value=F16, io=F16)),
        # many requests over an 8-bit head-major cache with a sliding window, some of them empty
        ("attend_window_200", attend_case(200, (0, 3000), 32, 4, 128, block=32, layout=HND, value=E4M3, window=1024, empty=4)),
        # a wave of 64 sessions over the 8-bit latent pool, 16 query heads on one latent head
        ("attend_latent_64", attend_case(64, (2048, 32768), 16, 1, 576, planes=1, v_dim=512, block=64, value=E4M3)),
    ]
    return [dict(c, name=n) for n, c in cases]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("slots", "append", "attend", "attend"))
    if op == "slots":
        n = log_int(rng, 1, 2000)
        new = rng.choice((1, log_int(rng, 2, max(2, min(32768, 4000000 // n)))))
        return slots_case(n, rng.choice((1, 8, 16, 24, 32, 64, 100, 128)), (0, log_int(rng, 1, 8192)), (1, new), rng.choice((0, 5, 30)))
    if op == "append":
        if rng.random() < 0.3:
            return append_case(log_int(rng, 1, 50000), log_int(rng, 1, 4096), 1, 576, planes=1, block=rng.choice((16, 64)),
                               value=rng.choice((BF16, E4M3)), padded=rng.choice((0, 3)))
        value = rng.choice((BF16, F16, E4M3))
        shards = rng.choice((1, 1, 2, 4))
        return append_case(log_int(rng, 1, 8192), log_int(rng, 1, 4096), shards * rng.choice((1, 2, 3)), rng.choice((64, 128)),
                           shards=shards, block=rng.choice((8, 16, 20, 64)), layout=rng.choice((NHD, HND)), value=value,
                           io=value if value != E4M3 else rng.choice((BF16, F16)), padded=rng.choice((0, 3)))
    if rng.random() < 0.3:
        hi = log_int(rng, 64, 32768)
        return attend_case(log_int(rng, 1, max(1, min(128, 1000000 // hi))), (0, hi), rng.choice((8, 16, 24, 32)), 1, 576, planes=1,
                           v_dim=512, block=rng.choice((16, 64)), value=rng.choice((BF16, E4M3)))
    value = rng.choice((BF16, F16, E4M3))
    shards = rng.choice((1, 1, 2, 4))
    heads = shards * rng.choice((1, 2))
    hi = log_int(rng, 16, 16384)
    n = log_int(rng, 1, max(1, min(256, 160000 // hi)))
    return attend_case(n, (rng.choice((0, 1, hi // 2)), hi), heads * rng.choice((1, 2, 4, 5, 7, 8, 12, 16)), heads,
                       rng.choice((64, 128)), shards=shards, block=rng.choice((8, 16, 20, 32, 64)), layout=rng.choice((NHD, HND)),
                       value=value, io=value if value != E4M3 else rng.choice((BF16, F16)),
                       window=rng.choice((0, 0, 0, 512)), empty=rng.choice((0, 0, 5)))


def work(case):
    if case["op"] == "slots":
        n, bs = case["n_reqs"], case["block"]
        new = n * (1 - case["idle"] / 100) * (case["new_lo"] + case["new_hi"]) / 2
        # lengths in, offsets and lengths out, a block id in and out per new block, a slot and a position per token
        return {"bytes": n * (4 + 4 + 8 + 4) + new / bs * 8 + new * 12, "flops": 4 * new}
    if case["op"] == "append":
        n = case["tokens"] * case["planes"] * case["heads"] * case["dim"]
        return {"bytes": n * (SIZE[case["io"]] + SIZE[case["value"]]) + 8 * case["tokens"], "flops": 2 * n if case["value"] == E4M3 else n}
    lo, hi = case["len_lo"], case["len_hi"]
    mean = (lo + hi) / 2                                             # lengths are spread evenly
    if 0 < case["window"] < hi:
        w = case["window"]
        mean = w - max(0, w - lo) ** 2 / 2 / max(1, hi - lo)
    tokens = case["n_reqs"] * (1 - case["empty"] / 100) * mean
    dim, v_dim = case["dim"], case["v_dim"] or case["dim"]
    per_token = case["planes"] * case["heads"] * dim * SIZE[case["value"]] + 4 / case["block"]
    per_req = case["q_heads"] * (dim * 2 + v_dim * 2 + 4) + 4
    return {"bytes": tokens * per_token + case["n_reqs"] * per_req, "flops": tokens * case["q_heads"] * 2 * (dim + v_dim)}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def normal(shape, dtype, gen, scale=1.0):
    """N(0, 1) values in the tensor's type; 8-bit codes stand for value / scale."""
    if dtype != torch.float8_e4m3fn:
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda").div_(scale).clamp_(-E4M3_MAX, E4M3_MAX).to(dtype)
    return out


def geometry(case, n_blocks):
    """The pool's counts: one layer of it."""
    return dict(n_layers=1, n_planes=case["planes"], n_shards=case["shards"], heads_per_shard=case["heads"] // case["shards"],
                head_dim=case["dim"], elem_bytes=SIZE[case["value"]], block_size=case["block"], layout=case["layout"],
                n_blocks=n_blocks)


def buffers(case, n_blocks, gen, scale):
    """One tensor per (plane, shard), in the pool's own layout."""
    hps = case["heads"] // case["shards"]
    inner = (case["block"], hps) if case["layout"] == NHD else (hps, case["block"])
    return [normal((n_blocks, *inner, case["dim"]), DTYPE[case["value"]], gen, scale) for _ in range(case["planes"] * case["shards"])]


class Geometry:
    def __init__(self, **counts):
        self.__dict__.update(counts)


def cache_of(case, geom, bufs, scales, q_heads):
    """The handle that a serving program keeps for its pool."""
    from disaggregated_prefill_decode_gb300 import kvx
    code = {BF16: kvx.KVX_BF16, F16: kvx.KVX_F16, E4M3: kvx.KVX_E4M3}
    return kvx.kvx_cache_create(kvx.Pool(Geometry(**geom), bufs), value_type=code[case["value"]], io_type=code[case["io"]],
                                n_q_heads=q_heads, v_dim=case.get("v_dim", 0), window=case.get("window", 0),
                                k_scale=scales[0], v_scale=scales[1])


def lengths(rng, n, lo, hi, share_without):
    """n lengths spread evenly over [lo, hi], some of them 0, in an order of the seed's."""
    x = np.floor(lo + (hi - lo + 1) * (np.arange(n) + 0.5) / n).astype(np.int32)
    some = np.arange(n) * share_without // 100
    x[np.flatnonzero(np.diff(some, prepend=0))] = 0
    return rng.permutation(x)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "slots":
        n, bs = case["n_reqs"], case["block"]
        ctx = lengths(rng, n, case["ctx_lo"], case["ctx_hi"], 0)
        new = lengths(rng, n, case["new_lo"], case["new_hi"], case["idle"])
        had = -(-ctx.astype(np.int64) // bs)
        need = -(-(ctx.astype(np.int64) + new) // bs)
        ids = rng.permutation(int(need.sum()) + 64).astype(np.int32)
        width = -(-(case["ctx_hi"] + case["new_hi"]) // bs)
        table = np.full((n, width), -1, np.int32)
        table[np.arange(width) < had[:, None]] = ids[:int(had.sum())]
        free = ids[int(had.sum()):]
        tokens = int(new.sum())
        state.update(ctx=dev(ctx), new=dev(new), free=dev(free), table=dev(table), width=width, tokens=tokens,
                     blocks=int((need - had).sum()), tok_off=torch.zeros(n + 1, dtype=torch.int64, device="cuda"),
                     slots=torch.zeros(max(tokens, 1), dtype=torch.int64, device="cuda"),
                     pos=torch.zeros(max(tokens, 1), dtype=torch.int32, device="cuda"),
                     seq_len=torch.zeros(n, dtype=torch.int32, device="cuda"),
                     result=torch.zeros(3, dtype=torch.int64, device="cuda"))
        return state
    f8 = case["value"] == E4M3
    scales = (float(np.float32(rng.uniform(0.012, 0.02))), float(np.float32(rng.uniform(0.012, 0.02)))) if f8 else (1.0, 1.0)
    if case["planes"] == 1:
        scales = (scales[0], scales[0])
    state["scales"] = scales
    if case["op"] == "append":
        n, bs = case["tokens"], case["block"]
        left, runs = n, []
        while left:                                                  # tokens of one request after another
            runs.append(min(left, case["run"]))
            left -= runs[-1]
        first = rng.integers(0, bs, len(runs))                       # each goes on inside its last block
        need = [-(-(f + r) // bs) for f, r in zip(first.tolist(), runs)]
        n_blocks = int(1.2 * sum(-(-(bs - 1 + r) // bs) for r in runs)) + 8
        order = rng.permutation(n_blocks)
        at, parts = 0, []
        for f, r, k in zip(first.tolist(), runs, need):
            t = f + np.arange(r)
            parts.append(order[at:at + k][t // bs].astype(np.int64) * bs + t % bs)
            at += k
        slots = np.concatenate(parts)
        slots[rng.random(n) < case["padded"] / 100] = -1
        bufs = buffers(case, n_blocks, gen, scales[0])
        # keys and values lie side by side in the projection's output
        both = normal((n, case["planes"], case["heads"], case["dim"]), DTYPE[case["io"]], gen)
        state.update(bufs=bufs, slots=dev(slots), k=both[:, 0], v=both[:, 1] if case["planes"] == 2 else None,
                     stride=case["planes"] * case["heads"] * case["dim"])
        q_heads = case["heads"]
    else:
        n, bs = case["n_reqs"], case["block"]
        lens = lengths(rng, n, case["len_lo"], case["len_hi"], case["empty"])
        need = -(-lens.astype(np.int64) // bs)
        n_blocks = int(1.2 * need.sum()) + 8
        width = max(int(need.max()), 1)
        table = np.full((n, width), -1, np.int32)
        table[np.arange(width) < need[:, None]] = rng.permutation(n_blocks)[:int(need.sum())]
        bufs = buffers(case, n_blocks, gen, scales[0])
        v_dim = case["v_dim"] or case["dim"]
        state.update(bufs=bufs, lens=dev(lens), table=dev(table), width=width,
                     q=normal((n, case["q_heads"], case["dim"]), DTYPE[case["io"]], gen),
                     out=torch.zeros((n, case["q_heads"], v_dim), dtype=DTYPE[case["io"]], device="cuda"),
                     lse=torch.zeros((n, case["q_heads"]), dtype=torch.float32, device="cuda"))
        q_heads = case["q_heads"]
    if own:
        state["cache"] = cache_of(case, geometry(case, n_blocks), bufs, scales, q_heads)
    return state


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"slots": own_slots, "append": own_append, "attend": own_attend}[op](state)
    return {"slots": plain_slots, "append": plain_append, "attend": plain_attend}[op](state)


def own_slots(s):
    from disaggregated_prefill_decode_gb300 import kvx
    kvx.kvx_slot_map(s["ctx"], s["new"], s["case"]["n_reqs"], s["case"]["block"], s["free"], s["free"].numel(), s["table"],
                     s["width"], s["width"], s["tokens"], s["tok_off"], s["slots"], s["pos"], s["seq_len"], s["result"])
    return s["tok_off"], s["slots"], s["pos"], s["seq_len"], s["table"], s["result"]


def own_append(s):
    from disaggregated_prefill_decode_gb300 import kvx
    kvx.kvx_cache_append(s["cache"], 0, s["k"], s["stride"], s["v"], s["stride"], s["slots"], s["case"]["tokens"])
    return s["bufs"]


def own_attend(s):
    from disaggregated_prefill_decode_gb300 import kvx
    c = s["case"]
    kvx.kvx_cache_attend(s["cache"], 0, s["q"], c["q_heads"] * c["dim"], s["table"], s["width"], s["width"], s["lens"], c["n_reqs"],
                         s["out"], c["q_heads"] * (c["v_dim"] or c["dim"]), s["lse"])
    return s["out"], s["lse"]


def plain_slots(s):
    n, bs = s["case"]["n_reqs"], s["case"]["block"]
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    row = torch.arange(n, device="cuda")
    s["tok_off"][1:] = torch.cumsum(new, 0)
    seq_len = ctx + new
    had, need = (ctx + bs - 1) // bs, (seq_len + bs - 1) // bs
    end = torch.cumsum(need - had, 0)
    r = torch.repeat_interleave(row, need - had, output_size=s["blocks"])
    k = torch.arange(s["blocks"], device="cuda")
    table[r, had[r] + k - (end - (need - had))[r]] = s["free"][k]
    r = torch.repeat_interleave(row, new, output_size=s["tokens"])
    pos = ctx[r] + torch.arange(s["tokens"], device="cuda") - s["tok_off"][r]
    s["slots"][:s["tokens"]] = table[r, pos // bs].long() * bs + pos % bs
    s["pos"][:s["tokens"]] = pos.int()
    s["seq_len"][:] = seq_len.int()
    s["result"][0] = s["tok_off"][n]
    s["result"][1] = end[n - 1]
    s["result"][2] = 0
    return s["tok_off"], s["slots"], s["pos"], s["seq_len"], table, s["result"]


def plain_append(s):
    c = s["case"]
    hps = c["heads"] // c["shards"]
    slots = s["slots"]
    keep = slots >= 0
    blk, at = (slots // c["block"])[keep], (slots % c["block"])[keep]
    for p, x in enumerate((s["k"], s["v"])[:c["planes"]]):
        x = x[keep]
        if c["value"] == E4M3:
            inverse = float(np.float32(1.0) / np.float32(s["scales"][p]))
            x = (x.float() * inverse).clamp(-E4M3_MAX, E4M3_MAX)
        x = x.to(DTYPE[c["value"]])
        for i in range(c["shards"]):
            buf, part = s["bufs"][p * c["shards"] + i], x[:, i * hps:(i + 1) * hps]
            buf, part = (buf.view(torch.uint8), part.contiguous().view(torch.uint8)) if c["value"] == E4M3 else (buf, part)
            if c["layout"] == NHD:
                buf[blk, at] = part
            else:
                buf[blk, :, at] = part
    return s["bufs"]


def gathered(s, plane, table, dtype):
    """[request][position][head][dim] of the blocks of a table, from every shard."""
    c = s["case"]
    parts = []
    for i in range(c["shards"]):
        x = s["bufs"][plane * c["shards"] + i][table].to(dtype)
        x = x.transpose(2, 3) if c["layout"] == HND else x           # [request][block][slot][head][dim]
        parts.append(x.reshape(x.shape[0], -1, *x.shape[3:]))
    return torch.cat(parts, 2) if len(parts) > 1 else parts[0]


def plain_attend(s):
    c = s["case"]
    v_dim, group = c["v_dim"] or c["dim"], c["q_heads"] // c["heads"]
    table = s["table"].long().clamp(min=0)
    q = s["q"].float().view(c["n_reqs"], c["heads"], group, c["dim"]) * (s["scales"][0] / math.sqrt(c["dim"]))
    k = gathered(s, 0, table, torch.float32)
    pos = torch.arange(k.shape[1], device="cuda")
    valid = pos < s["lens"][:, None]
    if c["window"]:
        valid &= pos >= s["lens"][:, None] - c["window"]
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).masked_fill(~valid[:, None, None], float("-inf"))
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(3, keepdim=True)
    v = k[..., :v_dim] if c["planes"] == 1 else gathered(s, 1, table, torch.float32)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) * s["scales"][1] / torch.where(total == 0, 1.0, total)
    s["out"].copy_(out.reshape(c["n_reqs"], c["q_heads"], v_dim))
    s["lse"].copy_((top + torch.log(total)).view(c["n_reqs"], c["q_heads"]))
    return s["out"], s["lse"]


# ------------------------------------------------------------------------------------------------
# the same in 64 bits
# ------------------------------------------------------------------------------------------------

def exact(case, seed):
    """Attention: one request at a time, softmax by its definition. Append: the values before their rounding."""
    if case["op"] == "slots":
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "append":
        outs = []
        hps = case["heads"] // case["shards"]
        slots = s["slots"].cpu().numpy()
        rows = np.flatnonzero(slots >= 0)
        tok, blk, at = dev(rows), dev(slots[rows] // case["block"]), dev(slots[rows] % case["block"])
        for p in range(case["planes"]):
            x = (s["k"], s["v"])[p][tok].double() / s["scales"][p]
            if case["value"] == E4M3:
                x = torch.clamp(x, -E4M3_MAX, E4M3_MAX)
            for i in range(case["shards"]):
                buf = s["bufs"][p * case["shards"] + i].double()
                for h in range(hps):
                    if case["layout"] == NHD:
                        buf[blk, at, h] = x[:, i * hps + h]
                    else:
                        buf[blk, h, at] = x[:, i * hps + h]
                outs.append(buf)
        return outs
    n, v_dim, group = case["n_reqs"], case["v_dim"] or case["dim"], case["q_heads"] // case["heads"]
    out = torch.zeros((n, case["q_heads"], v_dim), dtype=torch.float64, device="cuda")
    lse = torch.full((n, case["q_heads"]), float("-inf"), dtype=torch.float64, device="cuda")
    for r, length in enumerate(s["lens"].tolist()):
        first = max(0, length - case["window"]) if case["window"] else 0
        if length == 0:
            continue
        blocks = s["table"][r:r + 1, :-(-length // case["block"])].long()
        planes = [gathered(s, p, blocks, torch.float64)[0, first:length] * s["scales"][p] for p in range(case["planes"])]
        for h in range(case["heads"]):
            rows = slice(h * group, (h + 1) * group)
            scores = s["q"][r, rows].double() @ planes[0][:, h].T / math.sqrt(case["dim"])
            lse[r, rows] = torch.logsumexp(scores, 1)
            out[r, rows] = torch.softmax(scores, 1) @ planes[-1][:, h, :v_dim]
    return out, lse
