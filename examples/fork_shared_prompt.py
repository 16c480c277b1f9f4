"""Several answers to one prompt: a decode worker that shares the prompt's pages.

A prompt is appended once, its keys normed and rotated on their way into the cache. kvx_pages_fork makes a row for each
answer from it: full pages are shared, the partial last one is copied. A step, captured in a CUDA graph, finds the free pages
(kvx_pages_free), gives the new tokens their slots, and per layer rotates and appends them (kvx_cache_append_rotated) and
attends (kvx_cache_attend_shared, which reads a prompt once for all answers where there is enough to share). Half way some
answers end and others are forked again, and the pages in use are moved to the pool's front (kvx_pages_compact,
kvx_cache_copy). Every output is checked against attention over a cache kept on the side, every rotation against its formula.

    python examples/fork_shared_prompt.py [steps] [answers]
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import numpy as np
import torch

from disaggregated_prefill_decode_gb300 import kvx
from kvx_inputs import PoolGeom

LAYERS, KV_HEADS, Q_HEADS, DIM, BLOCK = 2, 2, 8, 128, 16
EPS = 1e-6


def rotated(x, weight, positions, freq):
    """The norm and rotation of heads [tokens][heads][dim] by their definition, in 64 bits."""
    x = x.double()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.double()
    angle = positions.double()[:, None, None] * freq
    a, b = x[..., :DIM // 2], x[..., DIM // 2:]
    return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)


def main(steps: int = 40, prompt: int = 500, answers: int = 12, seed: int = 0) -> tuple:
    """(largest error of an output, largest error of a rotated value over its size) against 64 bits."""
    torch.manual_seed(seed)
    n, width = answers, -(-(prompt + steps) // BLOCK)
    n_blocks = prompt // BLOCK + 3 * n * (steps // BLOCK + 2) + 50
    geom = PoolGeom(LAYERS, 2, 1, KV_HEADS, DIM, 2, BLOCK, n_blocks)
    bufs = [torch.empty(geom.buffer_bytes, dtype=torch.uint8, device="cuda") for _ in range(geom.n_buffers)]
    for b in bufs:
        b.view(torch.bfloat16).fill_(float("nan"))                         # unused slots may hold anything
    i32, i64 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int64, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    q_weight, k_weight = (1 + 0.2 * torch.randn(DIM, device="cuda")).bfloat16(), (1 + 0.2 * torch.randn(DIM, device="cuda")).bfloat16()
    cache = kvx.kvx_cache_create(kvx.Pool(geom, bufs), kvx.KVX_BF16, n_q_heads=Q_HEADS)
    turn = kvx.kvx_rotation_create(dim=DIM, scaling=kvx.KVX_ROTATE_BANDS, base=500000.0, factor=8.0, low=1.0, high=4.0, original=8192.0)
    freq = torch.from_numpy(kvx.kvx_rotation_get(turn)[0].copy()).cuda()
    side = torch.cuda.Stream()

    # what a model's projection would write: queries, keys and values of a token side by side
    row = (Q_HEADS + 2 * KV_HEADS) * DIM
    table, new_table = torch.full((n, width), -1, **i32), torch.full((n, width), -1, **i32)
    ctx, seq_len, new_len = torch.zeros(n, **i32), torch.zeros(n, **i32), torch.zeros(n, **i32)
    refs, free, result = torch.zeros(n_blocks, **i32), torch.zeros(n_blocks, **i32), torch.zeros(3, **i64)
    src, dst = torch.full((n_blocks,), -1, **i32), torch.full((n_blocks,), -1, **i32)
    first, parent = torch.zeros(n, **i32), torch.zeros(n, **i32)
    group_off, prefix_len = torch.tensor([0, n], **i32), torch.tensor([prompt], **i32)
    space = torch.empty(max(kvx.kvx_cache_shared_bytes(cache, n, 1), 16), dtype=torch.uint8, device="cuda")
    worst = [0.0, 0.0]

    def append(x, layer, q_out, positions, slots, tokens):
        q, k, v = x[:, :Q_HEADS * DIM], x[:, Q_HEADS * DIM:-KV_HEADS * DIM], x[:, -KV_HEADS * DIM:]
        kvx.kvx_cache_append_rotated(cache, layer, turn, q, row, q_weight, q_out, Q_HEADS * DIM, k, row, k_weight, v, row, positions,
                                     slots, tokens, side)

    def stored(layer, plane, slots):
        return bufs[layer * 2 + plane].view(torch.bfloat16).view(-1, KV_HEADS, DIM)[slots].double()

    def check_rotation(x, layer, q_out, positions, slots):
        heads = x.view(len(x), Q_HEADS + 2 * KV_HEADS, DIM)
        for got, want in ((q_out, rotated(heads[:, :Q_HEADS], q_weight, positions, freq)),
                          (stored(layer, 0, slots), rotated(heads[:, Q_HEADS:-KV_HEADS], k_weight, positions, freq))):
            worst[1] = max(worst[1], ((got.double() - want).abs() / (want.abs() + 1e-2)).max().item())
        assert torch.equal(stored(layer, 1, slots), heads[:, -KV_HEADS:].double())

    # the prompt: request 0, all of whose pages are taken from an empty pool
    free.copy_(torch.from_numpy(np.random.default_rng(seed).permutation(n_blocks).astype(np.int32)))
    lens = torch.zeros(n, **i32)
    lens[0] = prompt
    tok_off, slots, positions = torch.zeros(n + 1, **i64), torch.zeros(prompt, **i64), torch.zeros(prompt, **i32)
    x = torch.randn((LAYERS, prompt, row), device="cuda").bfloat16()
    q_out = torch.zeros((LAYERS, prompt, Q_HEADS, DIM), **bf16)
    torch.cuda.synchronize()
    kvx.kvx_slot_map(ctx, lens, n, BLOCK, free, n_blocks, table, width, width, prompt, tok_off, slots, positions, seq_len, result, side)
    for layer in range(LAYERS):
        append(x[layer], layer, q_out[layer], positions, slots, prompt)
    side.synchronize()
    kept = [[None] * n for _ in range(LAYERS)]                             # [layer][row]: keys and values
    for layer in range(LAYERS):
        check_rotation(x[layer], layer, q_out[layer], positions, slots)
        kept[layer][0] = [stored(layer, p, slots) for p in range(2)]

    def fork(parents):
        """The rows go on from these rows; their partial pages are copied in every layer."""
        nonlocal kept
        parent.copy_(torch.tensor(parents, **i32))
        free.fill_(-1)                                                     # behind the free pages: no page, not one of an earlier list
        torch.cuda.synchronize()
        kvx.kvx_pages_free(table, width, width, seq_len, n, BLOCK, n_blocks, refs, free, result, side)
        kvx.kvx_pages_fork(table, width, width, seq_len, n, parent, n, BLOCK, free, n, new_table, width, new_len, src, dst, first, result, side)
        kvx.kvx_cache_copy(cache, 0, LAYERS, src, dst, n, side)
        side.synchronize()
        assert result[2].item() == kvx.KVX_OK
        table.copy_(new_table)
        seq_len.copy_(new_len)
        kept = [[None if p < 0 else list(kept[layer][p]) for p in parents] for layer in range(LAYERS)]

    def compact():
        """Pages in use to the pool's front."""
        torch.cuda.synchronize()
        kvx.kvx_pages_free(table, width, width, seq_len, n, BLOCK, n_blocks, refs, free, result, side)
        kvx.kvx_pages_compact(table, width, width, seq_len, n, BLOCK, refs, n_blocks, table, width, src, dst, n_blocks, result, side)
        kvx.kvx_cache_copy(cache, 0, LAYERS, src, dst, n_blocks, side)
        side.synchronize()
        held, moved, status = result.tolist()
        assert status == kvx.KVX_OK and moved > 0
        cols = torch.arange(width, device="cuda") < (seq_len[:, None] + BLOCK - 1) // BLOCK
        assert torch.equal(table[cols].unique(), torch.arange(held, device="cuda", dtype=torch.int32))

    one = torch.ones(n, **i32)
    tok_off, slots, positions = torch.zeros(n + 1, **i64), torch.zeros(n, **i64), torch.zeros(n, **i32)
    x = torch.zeros((LAYERS, n, row), **bf16)
    q_out, out = torch.zeros((LAYERS, n, Q_HEADS, DIM), **bf16), torch.zeros((LAYERS, n, Q_HEADS, DIM), **bf16)

    def step():
        ctx.copy_(seq_len)
        free.fill_(-1)
        kvx.kvx_pages_free(table, width, width, ctx, n, BLOCK, n_blocks, refs, free, result, side)
        kvx.kvx_slot_map(ctx, one, n, BLOCK, free, n, table, width, width, n, tok_off, slots, positions, seq_len, result, side)
        for layer in range(LAYERS):
            append(x[layer], layer, q_out[layer], positions, slots, n)
            kvx.kvx_cache_attend_shared(cache, layer, q_out[layer], Q_HEADS * DIM, table, width, width, seq_len, n, group_off, prefix_len, 1,
                                        out[layer], Q_HEADS * DIM, None, space, space.numel(), side)

    fork([0] * n)
    graph = None
    for t in range(steps):
        if t == steps // 2:                                                # some answers end, others go on twice
            fork([int(p) for p in np.random.default_rng(1).integers(0, n // 2, n)])
            compact()
        x.normal_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            if t == 0:
                step()                                                     # the handle's scratch is there by now; the others replay one graph
            else:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=side):
                        step()
                graph.replay()
        torch.cuda.synchronize()
        assert result[2].item() == kvx.KVX_OK
        for layer in range(LAYERS):
            check_rotation(x[layer], layer, q_out[layer], positions, slots)
            for r in range(n):
                k, v = (torch.cat([kept[layer][r][p], stored(layer, p, slots[r:r + 1])]) for p in range(2))
                kept[layer][r] = [k, v]
                group = Q_HEADS // KV_HEADS
                kk, vv = (y.repeat_interleave(group, 1) for y in (k, v))
                p = torch.softmax(torch.einsum("hd,thd->ht", q_out[layer, r].double(), kk) / DIM ** 0.5, 1)
                worst[0] = max(worst[0], (torch.einsum("ht,thd->hd", p, vv) - out[layer, r].double()).abs().max().item())
    assert kvx.kvx_cache_status(cache) == kvx.KVX_OK
    kvx.kvx_cache_destroy(cache)
    kvx.kvx_rotation_destroy(turn)
    return tuple(worst)


if __name__ == "__main__":
    n_steps, n_answers = (int(sys.argv[i]) if len(sys.argv) > i else x for i, x in ((1, 40), (2, 12)))
    print("%d steps of %d answers, largest error of an output %.2g, of a rotated value %.2g of its size" %
          (n_steps, n_answers, *main(n_steps, answers=n_answers)))
