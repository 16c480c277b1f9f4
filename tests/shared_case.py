"""Batches whose requests share prefixes, for the tests of kvx_cache_attend_shared: tables in which the full pages of a prefix are the
same and the page that it ends in is a copy, checked by the same 64-bit statement as kvx_cache_attend."""
import numpy as np

import decode_reference as ref
from test_decode_gpu import Attend, dev, kvx, torch, typed, TYPES

# What two values leave of a weight and of the row's largest: bf16 first cut off, 2^-7, then half a unit, 2^-16 (and the lowest
# bit set, 2^-23); f16 2^-10, then cut off to an odd last place, a whole unit: 2^-20, its step 2^-24 of weights taken times 2^12 or more: 2^-35;
# f16 from 8-bit values both rounded: 2^-22, half a step: 2^-36.
PARTS = {"bf16": (2.0 ** -15.9, 0.0), "f16": (2.0 ** -20, 2.0 ** -35), "e4m3": (2.0 ** -22, 2.0 ** -36)}


class Shared(Attend):
    """groups: (prefix, [length of each member's rest], ...) or an int, a request alone. `say`: what prefix_len says, if not the
    prefix itself."""

    def __init__(self, groups, say=None, **kw):
        lens, off, prefix, alone = [], [0], [], []
        for g in groups:
            p, rest = (g if isinstance(g, tuple) else (0, [g]))
            lens += [p + x for x in rest]
            off.append(len(lens))
            prefix.append(p)
        super().__init__(lens, **kw)
        bs, layout = self.bs, self.geom.layout
        for i, p in enumerate(prefix):
            for r in range(off[i] + 1, off[i + 1]):
                whole = p // bs
                for b in self.bufs:                                        # what its own pages of the prefix held becomes NaN
                    raw = b.view(torch.uint8).view(self.geom.n_blocks, -1)
                    raw[dev(self.table[r, :whole].astype(np.int64))] = 0xFF
                self.table[r, :whole] = self.table[off[i], :whole]
                if p % bs:
                    src, dst = int(self.table[off[i], whole]), int(self.table[r, whole])
                    vdtype = TYPES[self.value][1]
                    for b in self.bufs:
                        v = typed(b, self.geom, vdtype).view(torch.uint8 if self.value == "e4m3" else torch.int16)
                        v[dst, :p % bs] = v[src, :p % bs]
                    for h in self.host:
                        h[dst * bs:dst * bs + p % bs] = h[src * bs:src * bs + p % bs]
        self.off, self.prefix = np.array(off, np.int32), np.array(prefix if say is None else say, np.int32)

    def shared(self, stream=None, pad=0, lse=True, max_blocks=None, off=None, prefix=None, lens=None):
        """As run. max_blocks is made so large that the batch is worth sharing; the table's rows end in garbage."""
        n, hq = len(self.lens), self.heads * self.group
        off, prefix = self.off if off is None else off, self.prefix if prefix is None else prefix
        again = max(1, n - min(len(prefix), n // 2))
        wide = max_blocks or max(self.width, (161 << 20) // (2 * self.geom.n_shards * self.geom.row_bytes * self.bs * again) + 2)
        table = np.full((n, wide), 2 ** 30, np.int32)
        table[:, :min(wide, self.table.shape[1])] = self.table[:, :wide]
        q = torch.zeros((n, hq * self.dim + pad), dtype=self.iodtype)
        q[:, :hq * self.dim] = self.q.reshape(n, -1)
        self.d_q, self.d_table = q.cuda(), dev(table)
        self.d_len = dev(np.array(self.lens if lens is None else lens, np.int32))
        self.d_off, self.d_prefix = dev(np.asarray(off, np.int32)), dev(np.asarray(prefix, np.int32))
        out = torch.full((n, hq * self.v_dim + pad), 7.0, dtype=self.iodtype, device="cuda")
        self.d_lse = torch.full((n, hq), 7.0, dtype=torch.float32, device="cuda")
        size = kvx.kvx_cache_shared_bytes(self.cache, n, len(prefix))
        self.space = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")        # NaN wherever nothing is written
        torch.cuda.synchronize()
        kvx.kvx_cache_attend_shared(self.cache, 0, self.d_q, q.shape[1], self.d_table, wide, wide, self.d_len, n, self.d_off, self.d_prefix,
                                    len(prefix), out, out.shape[1], self.d_lse if lse else None, self.space, size, stream)
        torch.cuda.synchronize()
        assert (self.space[size:] == 0xFF).all()
        if pad:
            assert (out[:, hq * self.v_dim:] == 7.0).all()
        return out[:, :hq * self.v_dim].reshape(n, hq, self.v_dim).clone(), self.d_lse.clone()

    def check_parts(self, out, lse, table=None):
        """Within the bounds of weights held in two values."""
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        table = self.table if table is None else table
        unit, step = PARTS[self.value]
        for r, n in enumerate(self.lens):
            first = max(0, n - self.window) if self.window else 0
            rows = ref.rows_of(table[r], np.arange(first, max(n, 0)), self.bs, self.geom.n_blocks)
            for h in range(self.heads):
                hs = slice(h * self.group, (h + 1) * self.group)
                k, v = self.host[0][rows, h], self.host[-1][rows, h, :self.v_dim]
                o, l, weight, spread, floor = ref.attend(self.q[r, hs].double().numpy(), k, v, self.scale)
                if len(rows) == 0:
                    assert (out[r, hs] == 0).all() and (lse[r, hs] == -np.inf).all(), (r, h)
                    continue
                score = (self.dim + 8) * 2.0 ** -24 * spread + 2.0 ** -20
                rel = 2 * score[:, None] + unit + (len(rows) + 64) * 2.0 ** -24
                err = rel * weight + step * floor
                b_out = ref.UNIT[self.io] * (np.abs(o) + err) + err + ref.SMALLEST[self.io]
                b_lse = score + (len(rows) + 64) * 2.0 ** -24 + np.abs(l) * 2.0 ** -22
                assert np.isfinite(out[r, hs]).all(), (r, h)
                off = np.abs(out[r, hs] - o) / b_out
                assert (off <= 1).all(), (r, h, n, off.max())
                off = np.abs(lse[r, hs] - l) / b_lse
                assert (off <= 1).all(), (r, h, n, off.max())


def check_shared(groups, **kw):
    case = Shared(groups, **kw)
    case.check_parts(*case.shared())
    assert kvx.kvx_cache_status(case.cache) == kvx.KVX_OK
    return case
