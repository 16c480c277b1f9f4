"""A decode worker's steps on the blocks that a push delivered.

A prefill pool (token-major, blocks of 16) is pushed layer by layer into a decode pool (head-major, blocks of 64).
The decode worker then takes steps of one token per request, each a CUDA graph replay: slots for the new tokens from
the requests' lengths, and per layer the append of their keys and values and their attention over the cache. At the
end every step's outputs are checked against the attention of a cache kept on the side.

    python examples/decode_after_push.py [steps]
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import numpy as np
import torch

from disaggregated_prefill_decode_gb300 import kvx
from kvx_inputs import LAYOUT_HND, PoolGeom

LAYERS, KV_HEADS, Q_HEADS, DIM = 2, 2, 8, 128


def buffers(geom, fill):
    made = [torch.empty(geom.buffer_bytes, dtype=torch.uint8, device="cuda") for _ in range(geom.n_buffers)]
    for b in made:
        fill(b.view(torch.bfloat16))
    return made


def main(steps: int = 70, lens=(37, 1, 700, 64), seed: int = 0) -> float:
    """Returns the largest error of an output against the check in 64 bits."""
    torch.manual_seed(seed)
    n = len(lens)
    src = PoolGeom(LAYERS, 2, 1, KV_HEADS, DIM, 2, 16, sum(-(-l // 16) for l in lens))
    spare = n * (steps // 64 + 2)
    dst = PoolGeom(LAYERS, 2, 1, KV_HEADS, DIM, 2, 64, sum(-(-l // 64) for l in lens) + spare, LAYOUT_HND)
    src_bufs = buffers(src, lambda t: t.normal_())
    dst_bufs = buffers(dst, lambda t: t.fill_(float("nan")))              # unused slots may hold anything

    # prefill -> decode: block ids on either side, one request after the other
    src_ids, dst_ids, at_s, at_d = [], [], 0, 0
    order = np.random.default_rng(seed).permutation(dst.n_blocks).astype(np.int32)
    for l in lens:
        src_ids.append(np.arange(at_s, at_s + -(-l // 16), dtype=np.int32))
        dst_ids.append(order[at_d:at_d + -(-l // 64)])
        at_s, at_d = at_s + -(-l // 16), at_d + -(-l // 64)
    side = torch.cuda.Stream()
    decode_pool = kvx.Pool(dst, dst_bufs)
    with kvx.kvx_plan(kvx.Pool(src, src_bufs), decode_pool, [(l, s, d) for l, s, d in zip(lens, src_ids, dst_ids)]) as plan:
        torch.cuda.synchronize()
        for layer in range(LAYERS):
            kvx.kvx_push_layer(plan, layer, side)
        assert kvx.kvx_sync(plan) == kvx.KVX_OK

    # the same keys and values on the side, for the check: [layer][plane][request] -> [tokens][heads][dim]
    kept = [[[src_bufs[layer * 2 + p].view(torch.bfloat16).view(-1, KV_HEADS, DIM)[int(s[0]) * 16:][:l].clone()
              for l, s in zip(lens, src_ids)] for p in range(2)] for layer in range(LAYERS)]

    width = max(-(-(l + steps) // 64) for l in lens)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((n, width), -1, **i32)
    for r, d in enumerate(dst_ids):
        table[r, :len(d)] = torch.from_numpy(d.copy())
    ctx, seq_len = torch.tensor(lens, **i32), torch.zeros(n, **i32)
    one = torch.ones(n, **i32)
    all_free = torch.from_numpy(np.concatenate([order[at_d:], np.zeros(n, np.int32)])).cuda()
    taken, ahead = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.arange(n, device="cuda")
    free = all_free[:n].clone()                                            # a step takes n blocks at most
    tok_off, slots = torch.zeros(n + 1, dtype=torch.int64, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")
    result = torch.zeros(3, dtype=torch.int64, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((LAYERS, n, Q_HEADS, DIM), **bf16)                     # what a model's projections would write
    kv = torch.zeros((LAYERS, 2, n, KV_HEADS, DIM), **bf16)
    out = torch.zeros((LAYERS, n, Q_HEADS, DIM), **bf16)
    cache = kvx.kvx_cache_create(decode_pool, kvx.KVX_BF16, n_q_heads=Q_HEADS)

    def step():
        kvx.kvx_slot_map(ctx, one, n, 64, free, n, table, width, width, n, tok_off, slots, None, seq_len, result, side)
        for layer in range(LAYERS):
            kvx.kvx_cache_append(cache, layer, kv[layer, 0], KV_HEADS * DIM, kv[layer, 1], KV_HEADS * DIM, slots, n, side)
            kvx.kvx_cache_attend(cache, layer, q[layer], Q_HEADS * DIM, table, width, width, seq_len, n, out[layer], Q_HEADS * DIM,
                                 None, side)

    def next_step():
        ctx.copy_(seq_len)
        taken.add_(result[1:2])
        torch.index_select(all_free, 0, ahead + taken, out=free)

    # the first step makes the cache's scratch; the others replay one graph
    worst = 0.0
    graph = None
    for t in range(steps):
        q.normal_()
        kv.normal_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            if t == 0:
                step()
                next_step()
            else:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=side):
                        step()
                        next_step()
                graph.replay()
        torch.cuda.synchronize()
        assert result[2].item() == kvx.KVX_OK
        for layer in range(LAYERS):
            for r in range(n):
                k, v = (torch.cat([kept[layer][p][r], kv[layer, p, r:r + 1]]) for p in range(2))
                kept[layer][0][r], kept[layer][1][r] = k, v
                group = Q_HEADS // KV_HEADS
                kk, vv = (x.double().repeat_interleave(group, 1) for x in (k, v))
                p = torch.softmax(torch.einsum("hd,thd->ht", q[layer, r].double(), kk) / DIM ** 0.5, 1)
                worst = max(worst, (torch.einsum("ht,thd->hd", p, vv) - out[layer, r].double()).abs().max().item())
    assert kvx.kvx_cache_status(cache) == kvx.KVX_OK
    kvx.kvx_cache_destroy(cache)
    return worst


if __name__ == "__main__":
    n_steps = int(sys.argv[1]) if len(sys.argv) > 1 else 70
    print(f"{n_steps} steps after the push, largest error of an output {main(n_steps):.2g}")
