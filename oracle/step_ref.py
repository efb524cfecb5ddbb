"""Plain restatements of the operators around a model's blocks (numpy, Python integers).

``kv_step`` walks the requests one after another, ``sample_row`` the sorted tokens of one row;
``embed_grad`` is the formula in fp64.  No code is shared with the GPU path.
"""
from __future__ import annotations

import numpy as np

F = np.float32


def kv_step(cached, fresh, blocks, free, count, page, T):
    """(seq, pos, slot, lens, starts, count); blocks and free are updated in place."""
    B, per = blocks.shape
    count = min(max(int(count), 0), len(free))
    for b in range(B):                       # ended requests give their pages back
        if fresh[b] < 0:
            for i in range(min(-(-max(int(cached[b]), 0) // page), per)):
                if count < len(free):
                    free[count] = blocks[b, i]
                    count += 1
    room, pages_wanted, rows_wanted = count, 0, 0
    seq, pos, slot = (np.full(T, -1, d) for d in (np.int32, np.int32, np.int64))
    lens, starts = np.zeros(B, np.int32), np.zeros(B + 1, np.int32)
    t = 0
    for b in range(B):
        n, f = max(int(cached[b]), 0), int(fresh[b])
        starts[b] = t
        if f >= 0:
            have, need = -(-n // page), -(-(n + f) // page)
            pages_wanted += need - have
            rows_wanted += f
            if (need <= per and (need == have or pages_wanted <= room) and rows_wanted <= T and
                    n + f < 2 ** 31):
                for i in range(have, need):
                    count -= 1
                    blocks[b, i] = free[count]
                for p in range(n, n + f):
                    seq[t], pos[t], slot[t] = b, p, int(blocks[b, p // page]) * page + p % page
                    t += 1
                n += f
            lens[b] = n
    starts[B] = t
    return seq, pos, slot, lens, starts, count


def embed(ids, table, scale):
    """fp32 rows before their rounding."""
    V = len(table)
    y = np.zeros((len(ids), table.shape[1]), F)
    for t, v in enumerate(ids):
        y[t] = 0.0 if v < 0 else np.nan if v >= V else np.asarray(table[v], F) * F(scale)
    return y


def embed_grad(dy, ids, V, scale, into=None):
    """(dtable in fp64, sums of magnitudes, tokens per row)."""
    dy = np.asarray(dy, np.float64)
    ok = (ids >= 0) & (ids < V)
    out, mag = np.zeros((V, dy.shape[1])), np.zeros((V, dy.shape[1]))
    np.add.at(out, ids[ok], dy[ok] * scale)
    np.add.at(mag, ids[ok], np.abs(dy[ok] * scale))
    if into is not None:
        out, mag = out + into, mag + np.abs(into)
    return out, mag, np.bincount(ids[ok], minlength=V)
