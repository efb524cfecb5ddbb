"""Plain restatements of the operators between a decoder block's projections (numpy).

``norm_quant`` and ``rope`` follow the fp32 operations of the definition one by one (their results
are defined to the bit: separate fp32 products and sums, the mean square summed exactly), so they
pin the int8 rows and the rotated values exactly.  ``norm_grad`` and ``paged_attn`` are the formulas
in fp64.  No code is shared with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

from .bitlinear_ref import act_quant

F = np.float32


def bf16_round(x):
    """fp32 values rounded to the nearest bfloat16 (ties to even), as fp32."""
    u = np.ascontiguousarray(x, F).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32) << 16).view(F).reshape(np.shape(x))


def norm_quant(x, w=None, res=None, eps=1e-6, lift_M=0, res_bf16=False):
    """(xq, scale, h, rstd) of fp32 arrays x[T][K], res[T][K], w[K]."""
    h = np.asarray(x, F)
    if res is not None:
        h = h + np.asarray(res, F)
        if res_bf16:
            h = bf16_round(h)
    sq = h * h
    K = h.shape[1]
    rstd = np.array([F(1.0 / math.sqrt(math.fsum(float(v) for v in row) / K + eps)) for row in sq],
                    F).reshape(-1)
    n = h * rstd[:, None]
    if w is not None:
        n = n * np.asarray(w, F)
    xq, scale = act_quant(n, lift_M)
    return xq, scale, h, rstd


def norm_rows(h, w, eps):
    """The normed rows in fp64."""
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def norm_grad(dn, h, rstd, w, dres=None):
    """(dh, dw) in fp64 from the formula, at the given rstd."""
    dn, h, r, w = (np.asarray(v, np.float64) for v in (dn, h, rstd, w))
    nh = h * r[:, None]
    gw = dn * w
    dh = r[:, None] * (gw - nh * (gw * nh).mean(-1, keepdims=True))
    if dres is not None:
        dh = dh + np.asarray(dres, np.float64)
    return dh, (dn * nh).sum(0)


def rope_table(freq, positions, mscale=1.0):
    a = np.arange(positions, dtype=np.float64)[:, None] * np.asarray(freq, np.float64)
    return np.stack((np.cos(a) * mscale, np.sin(a) * mscale), -1).astype(F)


def rope(x, pos, table, interleaved=False, inverse=False):
    """fp32 x[T][H][D]; padding positions give 0, positions past the table NaN."""
    x = np.asarray(x, F)
    half = table.shape[1]
    y = x.copy()
    for t, p in enumerate(pos):
        if p < 0 or p >= len(table):
            y[t] = 0.0 if p < 0 else np.nan
            continue
        c, s = table[p, :, 0], table[p, :, 1]
        if inverse:
            s = -s
        ia, ib = ((np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if interleaved
                  else (np.arange(half), np.arange(half, 2 * half)))
        a, b = x[t][:, ia], x[t][:, ib]
        y[t][:, ia] = a * c - b * s
        y[t][:, ib] = b * c + a * s
    return y


def paged_attn(q, kc, vc, blocks, lens, scale, window=0, ks=None, vs=None):
    """out[B][Hq][D], lse[B][Hq] and absolute sums in fp64; caches [pages][heads][page][D].

    The third result is sum_j p_j |v_j| and the fourth max_j sum_d |q_d k_jd| * |scale|, which error
    bounds are made of.
    """
    B, Hq, D = q.shape
    pages, heads, ps, _ = kc.shape
    G = Hq // heads
    out, mag = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, smag = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    for b in range(B):
        n = max(0, min(int(lens[b]), blocks.shape[1] * ps))
        t = np.arange(max(0, n - window) if window else 0, n)
        pg = blocks[b, t // ps] if n else np.zeros(0, int)
        ok = (pg >= 0) & (pg < pages)
        pg, off = pg[ok], t[ok] % ps
        if not len(pg):
            continue
        for h in range(heads):
            k, v = kc[pg, h, off].astype(np.float64), vc[pg, h, off].astype(np.float64)
            if ks is not None:
                k = k * ks[pg, h, off].astype(np.float64)[:, None]
                v = v * vs[pg, h, off].astype(np.float64)[:, None]
            for j in range(h * G, (h + 1) * G):
                row = q[b, j].astype(np.float64)
                s = k @ row * scale
                m = s.max()
                if m == -np.inf:      # every weight is zero
                    continue
                p = np.exp(s - m)
                out[b, j] = p @ v / p.sum()
                mag[b, j] = p @ np.abs(v) / p.sum()
                lse[b, j] = m + np.log(p.sum())
                smag[b, j] = (np.abs(k) @ np.abs(row)).max() * abs(scale)
    return out, lse, mag, smag
