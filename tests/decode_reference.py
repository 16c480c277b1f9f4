"""Plain statements of the decode side in Python and 64 bits, with the error bounds its 16- and 32-bit
arithmetic allows: slot maps by loops, attention one request and head at a time by its definition."""
from __future__ import annotations

import numpy as np

# half a unit in the last place, relative: rounding to the type
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def slot_map(ctx, new, bs, free, table, max_blocks, max_tokens):
    """(tok_off, slots, positions, seq_len, table, n_tokens, n_blocks, status) as kvx_slot_map defines them."""
    ok, erange, enomem = 0, 2, 5
    table = table.copy()
    tok_off, slots, pos, seq, taken, bad = [0], [], [], [], 0, False
    for r, (c, n) in enumerate(zip(ctx.tolist(), new.tolist())):
        bad |= c < 0 or n < 0
        c, n = max(c, 0), max(n, 0)
        if c + n > 2 ** 31 - 1:
            bad, n = True, 2 ** 31 - 1 - c
        had, need = -(-c // bs), -(-(c + n) // bs)
        bad |= need > max_blocks
        for j in range(min(had, max_blocks), min(need, max_blocks)):
            table[r, j] = free[taken] if taken < len(free) else -1
            taken += 1
        if n and c % bs and c // bs < max_blocks:
            bad |= table[r, c // bs] < 0
        for t in range(c, c + n):
            blk = int(table[r, t // bs]) if t // bs < max_blocks else -1
            slots.append(blk * bs + t % bs if blk >= 0 else -1)
            pos.append(t)
        tok_off.append(tok_off[-1] + n)
        seq.append(c + n)
    total = tok_off[-1]
    bad |= total > max_tokens
    out = np.full(max_tokens, -1, np.int64)
    out[:min(total, max_tokens)] = slots[:max_tokens]
    return (np.array(tok_off, np.int64), out, np.array(pos[:max_tokens], np.int32), np.array(seq, np.int32), table, total,
            taken, enomem if taken > len(free) else erange if bad else ok)


def rows_of(table_row, positions, bs, n_blocks):
    """Pool rows (block * bs + slot) of the positions whose block lies in the pool."""
    blk = table_row[positions // bs].astype(np.int64)
    keep = (blk >= 0) & (blk < n_blocks)
    return blk[keep] * bs + positions[keep] % bs


def attend(q, k, v, scale):
    """One head: (out, lse, and the sums the bounds need). q: [group][d], k: [n][d], v: [n][dv], float64, already scaled."""
    if len(k) == 0:
        g = len(q)
        return np.zeros((g, v.shape[1])), np.full(g, -np.inf), np.zeros((g, v.shape[1])), np.zeros(g), np.zeros((g, v.shape[1]))
    s = q @ k.T * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(1, keepdims=True)
    spread = (np.abs(q) @ np.abs(k).T).max(1) * abs(scale)                # largest sum of |q_i k_i|
    return (p @ v / total, (m + np.log(total))[:, 0], p @ np.abs(v) / total, spread, np.abs(v).sum(0) / total)


def attend_bounds(out, lse, weight, spread, floor, d, n, io, p_unit):
    """Bounds of |out - exact| and |lse - exact| for 32-bit sums of exact products, weights rounded to p_unit, outputs to io.
    Scores: d products and a scaling summed in 32 bits, each step off by 2^-24 of at most `spread`, a query rounded 2^-24 of its
    row's largest element, 2^-20 for the exponential; a weight's relative error is its score's. Weights: p_unit each (and 2^-25 of
    the largest weight where they underflow), n of them and their sums in 32 bits, in up to four stages."""
    score = (d + 8) * 2.0 ** -24 * spread + 2.0 ** -20
    rel = 2 * score[:, None] + p_unit + (n + 64) * 2.0 ** -24
    bound_out = UNIT[io] * (np.abs(out) + rel * weight) + rel * weight + 2.0 ** -25 * floor * (1 if p_unit else 0) + 2.0 ** -24
    bound_lse = score + (n + 64) * 2.0 ** -24 + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -22
    return bound_out, bound_lse


# ------------------------------------------------------------------------------------------------
# bounds for weights held in parts
# ------------------------------------------------------------------------------------------------

# What the parts of a weight leave of it, at most: relative to the weight, and (small ones) relative to the row's largest.
#   bf16, two values: the second takes what truncation left, below 2^-7, and is half a unit of its own off: 2^-16. No floor.
#   bf16, three values: the second is cut off too, 2^-14, and the third is 2^-8 off: 2^-22. No floor.
#   f16, two values: below 2^-10, then half a unit: 2^-22. The second's smallest step is 2^-24 of weights taken times 2^15
#     (2^12 on the tensor pipe), and may be a whole step off: 2^-39 (2^-36).
#   e4m3, N codes 2^5 apart: each leaves 2^-4 of the power of two below what it stands for, 2^-4-5(N-1) in all; the last
#     one's smallest step is 2^-9 of weights taken times 2^5, half of it 2^-10-5N. Of four the last two are taken from an f16
#     value, 2^-11 off where the last code is 2^-9: a quarter more of each, and 2^-18 for 2^-19.
#   e4m3, four codes 1, 2^10 and 2^5 apart (the second is of the first one's scale): the same of large weights and of the smallest.
#     Between, the first two end at half their step, 2^-10 of weights taken times 2^5, and the other two leave 2^-4-5 of that (the
#     second of them half a step, where a power of two ends: 2^-10), or of a weight that is smaller.
PARTS = {"bf16": (2.0 ** -16, 0.0), "bf16 planes": (2.0 ** -22, 0.0), "f16": (2.0 ** -22, 2.0 ** -39), "f16 tensor": (2.0 ** -22, 2.0 ** -36),
         "3 codes": (2.0 ** -14, 2.0 ** -25), "4 codes": (2.0 ** -18, 1.25 * 2.0 ** -30),
         "4 codes, wide": (2.0 ** -18, 1.25 * 2.0 ** -30, 1.25 * 2.0 ** -9, 1.25 * 2.0 ** -25)}
SMALLEST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}                       # half an output's smallest step


def parts_bounds(out, lse, weight, spread, floor, d, n, io, parts):
    """As attend_bounds, for weights that are held in parts."""
    unit, step = PARTS[parts][:2]
    low_unit, low_step = PARTS[parts][2:] or (0.0, 0.0)
    score = (d + 8) * 2.0 ** -24 * spread + 2.0 ** -20
    rel = 2 * score[:, None] + unit + (n + 64) * 2.0 ** -24
    err = rel * weight + step * floor + np.minimum(low_unit * weight, low_step * floor)
    return UNIT[io] * (np.abs(out) + err) + err + SMALLEST[io], score + (n + 64) * 2.0 ** -24 + np.abs(lse) * 2.0 ** -22


def paired_values(rng, n, heads, dim, spread):
    """Keys of nearly equal scores and values in pairs of opposite sign: outputs are small differences of large sums, so that
    a weight's rounding shows beside the output's. keys, values [n][heads][dim]."""
    k = rng.standard_normal((n, heads, dim)) * spread
    half = rng.standard_normal(((n + 1) // 2, heads, dim))
    return k, np.stack([half, -half], 1).reshape(-1, heads, dim)[:n]


def one_large_score(rng, n, heads, dim, gap, scale, q0, size):
    """One position whose score is `gap` above the others' and whose value is nearly nothing, as the first token's often is.
    The gap comes from element 0 of the queries, q0. keys, values [n][heads][dim]."""
    k = rng.standard_normal((n, heads, dim)) * 0.5
    v = (np.abs(rng.standard_normal((n, heads, dim))) + 0.5) * size
    at = n // 3
    k[:, :, 0] = 0
    k[at] = 0
    k[at, :, 0] = gap / (q0 * scale)
    v[at] = 0
    return k, v
