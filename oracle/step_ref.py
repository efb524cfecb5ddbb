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


def bf16_bits(x):
    """Bit patterns of fp32 values that bfloat16 holds."""
    return (np.ascontiguousarray(x, F).view(np.uint32) >> 16).astype(np.uint16)


def q4_quantize(W, group):
    """(q int8 [n][K], s fp32 [n][K / group]) of fp32 weights; groups with an infinity or a NaN: 0, NaN."""
    from .block_ref import bf16_round
    n, K = W.shape
    w = np.asarray(W, F).reshape(n, K // group, group)
    amax = np.abs(w).max(-1)                 # NaN if there is one
    ok = np.isfinite(amax)
    s = np.where(ok, bf16_round(np.where(ok, amax, F(0)) / F(7)), F(np.nan)).astype(F)
    live = ok & (s > 0)
    with np.errstate(all="ignore"):
        r = np.rint(w / np.where(live, s, F(1))[..., None])
    q = np.where(live[..., None], np.clip(r, -7, 7), 0)
    return q.astype(np.int8).reshape(n, K), s


def q4_pack(q, s, group):
    """The documented layout, element by element: (codes uint8, scales uint16)."""
    n, K = q.shape
    NB, nt = -(-K // 128), -(-n // 16)
    qp = np.zeros((nt * 16, NB * 128), np.uint8)
    qp[:n, :K] = q.astype(np.uint8) & 15
    sp = np.zeros((nt * 16, NB * 128 // group), np.uint16)
    sp[:n, :K // group] = bf16_bits(s)
    sp[:n, :K // group][np.isnan(s)] = 0x7FC0
    codes = np.zeros((nt, NB, 64, 4, 4), np.uint8)
    scales = np.zeros((nt, NB, 4, 128 // group, 4), np.uint16)
    for l in range(64):
        h = l // 16
        for w in range(4):
            c = 32 * w + 8 * h if group == 32 else 64 * (w // 2) + 16 * h + 8 * (w % 2)
            for j in range(4):
                lo, hi = qp[l % 16::16, c + j::128], qp[l % 16::16, c + 4 + j::128]
                codes[:, :, l, w, j] = lo | hi << 4
    for h in range(4):
        for g in range(128 // group):
            for r in range(4):
                scales[:, :, h, g, r] = sp[4 * h + r::16, g::128 // group]
    return codes.reshape(-1), scales.reshape(-1)


def q4_forward(xq, x_scale, q, s, group):
    """(y, sum over groups of magnitudes) in fp64."""
    n, K = q.shape
    x = np.asarray(xq, np.float64).reshape(len(xq), K // group, group)
    w = np.asarray(q, np.float64).reshape(n, K // group, group)
    y, mag = (np.zeros((len(xq), n)) for _ in range(2))
    for g in range(K // group):
        part = (x[:, g] @ w[:, g].T) * np.asarray(s[:, g], np.float64)
        y += part
        mag += np.abs(part)
    xs = np.asarray(x_scale, np.float64)[:, None]
    return y * xs, mag * xs


def sample_row(x, u, temperature=1.0, k=0, p=1.0, min_p=0.0):
    """(token, log probability, its sum of p_i |x_i - top|) of one row, by walking down its tokens."""
    x = np.asarray(x, np.float64) + 0.0
    x = np.where(np.isnan(x), -np.inf, x)
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    top = x[order[0]]
    if top == -np.inf:
        return -1, -np.inf, 0.0
    d = np.where(x == top, 0.0, np.where(np.isinf(x) | (top == np.inf), -np.inf, x - (0 if top == np.inf else top)))
    e = np.exp(d)
    token = order[0]
    if temperature > 0:
        with np.errstate(all="ignore"):
            z = np.where(d == 0, 0.0, np.where(d == -np.inf, d, d / np.float64(temperature)))
        w = [int(v) for v in np.rint(np.exp(z) * 2.0 ** 40)]
        left = order[:k] if 0 < k < len(order) else order
        p = 1.0 if not p < 1 else max(float(p), 0.0)
        goal, total = p * float(sum(w[i] for i in left)), 0
        for n, i in enumerate(left):
            if n and (p < 1 and float(total) >= goal or min_p > 0 and float(w[i]) < float(min_p) * 2.0 ** 40):
                break
            total += w[i]
        r = min(int(min(u, 1.0) * float(total)) if u > 0 else 0, total - 1)
        for i in left:
            r -= w[i]
            if r < 0:
                token = i
                break
    live = e > 0
    return token, d[token] - np.log(e.sum()), float((e[live] * -d[live]).sum() / e.sum())
