"""Plain statements of the calls on pages, by loops over rows and blocks."""
from __future__ import annotations

import numpy as np

OK, ERANGE, ENOMEM = 0, 2, 5


def held(table, lens, bs):
    """Each row's blocks by its length, and whether a length was out of range."""
    cap = table.shape[1] * bs
    bad = bool(np.any((lens < 0) | (lens > cap)))
    cut = np.clip(lens.astype(np.int64), 0, cap)
    return [table[r, :-(-int(n) // bs)].tolist() for r, n in enumerate(cut)], cut.astype(np.int32), bad


def free(table, lens, bs, n_blocks):
    """(refs, free ids, result)"""
    rows, _, bad = held(table, lens, bs)
    refs = np.zeros(n_blocks, np.int32)
    for row in rows:
        for b in row:
            if 0 <= b < n_blocks:
                refs[b] += 1
            else:
                bad = True
    ids = np.flatnonzero(refs == 0).astype(np.int32)
    return refs, ids, [n_blocks - len(ids), len(ids), ERANGE if bad else OK]


def fork(table, lens, bs, parent, free_ids):
    """(new_table, new_len, src, dst, result)"""
    rows, cut, _ = held(table, lens, bs)
    cap = table.shape[1] * bs
    n_out = len(parent)
    new, new_len = np.full((n_out, table.shape[1]), -1, np.int32), np.zeros(n_out, np.int32)
    src, dst = np.full(n_out, -1, np.int32), np.full(n_out, -1, np.int32)
    seen, taken, bad, total = set(), 0, False, 0
    for i, p in enumerate(parent.tolist()):
        if not 0 <= p < len(rows):
            bad |= p != -1
            continue
        bad |= lens[p] < 0 or lens[p] > cap
        new[i, :len(rows[p])] = rows[p]
        new_len[i] = cut[p]
        total += len(rows[p])
        if cut[p] % bs and p in seen:
            if rows[p][-1] < 0:
                bad = True
            else:
                if taken < len(free_ids):
                    to = int(free_ids[taken])
                    bad |= to < 0
                    if to >= 0:
                        src[taken], dst[taken] = rows[p][-1], to
                    new[i, len(rows[p]) - 1] = max(to, -1)
                else:
                    new[i, len(rows[p]) - 1] = -1
                taken += 1
        seen.add(p)
    return new, new_len, src, dst, [total, taken, ENOMEM if taken > len(free_ids) else ERANGE if bad else OK]


def compact(table, lens, bs, refs, max_moves):
    """(new_table, pairs, result)"""
    rows, _, bad = held(table, lens, bs)
    n_blocks = len(refs)
    live = refs > 0
    n = int(live.sum())
    moves = list(zip(np.flatnonzero(live[n:]) + n, np.flatnonzero(~live[:n])))
    new = table.copy()
    fits = len(moves) <= max_moves
    to = dict((int(a), int(b)) for a, b in moves)
    for r, row in enumerate(rows):
        for j, b in enumerate(row):
            if not 0 <= b < n_blocks:
                bad = True
            elif fits and b >= n:
                if b in to:
                    new[r, j] = to[b]
                else:
                    bad = True
    return new, moves if fits else [], [n, len(moves), ENOMEM if not fits else ERANGE if bad else OK]
