"""Rotary positions and the append to a paged cache against plain implementations.

Every output is one rounded fp32 product or sum after another, so results equal the reference to the
bit: layouts, part of the head, strides, types, padding, and what the cache then holds.
"""
import numpy as np
import pytest

import oracle as O
import oracle.block_ref as R
from parity_util import bf16_dev, dev, f32_bits, host
from synth import rng, to_bf16

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")


def _t(g, shape, dtype):
    x = g.standard_normal(shape).astype(np.float32)
    if dtype == "bf16":
        x, bits = to_bf16(x)
        return x, bf16_dev(bits)
    return x, dev(x)


def _f32(t):
    return host(t.float())


def _same(a, b):
    a, b = np.ascontiguousarray(a), np.ascontiguousarray(b)
    ok = np.isnan(a) & np.isnan(b)
    return np.array_equal(f32_bits(np.where(ok, 0, a)), f32_bits(np.where(ok, 0, b)))


@pytest.mark.parametrize("T,heads,D,Rt", [(1, (20, 5), 128, 128), (37, (3, 1), 80, 32),
                                          (5, (1, 2), 96, 48), (300, (7,), 64, 64), (2, (4, 4, 4, 4), 256, 256),
                                          (9, (2, 2), 100, 100), (4, (3,), 33, 20), (6, (2, 1), 8, 8),
                                          (3, (2,), 2, 2), (1500, (2, 1), 72, 40)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("xd,yd", [("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_rope_equals_definition(T, heads, D, Rt, inter, xd, yd):
    import torch
    g = rng(T + D)
    P = 50 + T
    table = R.rope_table(S.rope_frequencies(Rt)[0], P)
    pos = g.integers(0, P, T).astype(np.int32)
    if T > 2:
        pos[0], pos[1] = -1, P                    # padding; a position without a table entry
    xs = [_t(g, (T, h, D), xd) for h in heads]
    dt = torch.bfloat16 if yd == "bf16" else torch.float32
    for inverse in (False, True):
        ys = S.rope([t for _, t in xs], dev(pos), dev(table), inter, inverse, dt)
        for (x, _), y in zip(xs, ys):
            want = R.rope(x, pos, table, inter, inverse)
            ok = ~np.isnan(want)
            if yd == "bf16":
                want = np.where(ok, R.bf16_round(np.where(ok, want, 0)), np.nan)
            assert y.dtype == dt and _same(_f32(y), want)


def test_rope_table_is_the_rounded_64_bit_value():
    for scaling in ("none", "linear", "base", "parts"):
        f, m = S.rope_frequencies(64, 10000.0, 1.0 if scaling == "none" else 8.0, scaling)
        got = host(S.rope_table(70001, f, m))
        want = R.rope_table(f, 70001, m)
        # both are correctly rounded up to a 64-bit error of a few 2^-53 in 2^-24: at most one unit
        # apart, at values that lie within that of a rounding boundary
        d = np.abs(got.astype(np.float64) - want)
        assert np.all(d <= 2.0 ** -23 * np.abs(want) + 1e-15) and np.mean(d > 0) < 1e-5


def test_rope_slices_in_place_and_inverse():
    """Heads as slices of a fused projection's rows, tokens-last storage, broadcast rows, in place;
    turning back gives the input up to the rounding of two rotations."""
    import torch
    g = rng(5)
    T, D = 19, 64
    table = dev(R.rope_table(S.rope_frequencies(64)[0], 64))
    pos = dev(g.integers(0, 64, T).astype(np.int32))
    x, qkv = _t(g, (T, 9, D), "f32")
    q, k = S.rope([qkv[:, :5], qkv[:, 5:7]], pos, table)
    want = R.rope(x, host(pos), host(table))
    assert _same(_f32(q), want[:, :5]) and _same(_f32(k), want[:, 5:7])
    by_head = qkv[:, :5].transpose(0, 1).contiguous().transpose(0, 1)
    assert _same(_f32(S.rope([by_head], pos, table)[0]), want[:, :5])
    one = qkv[:1, :1].expand(T, 5, D)
    assert _same(_f32(S.rope([one], pos, table)[0]),
                 R.rope(np.broadcast_to(x[:1, :1], (T, 5, D)), host(pos), host(table)))
    back = S.rope([q], pos, table, inverse=True)[0]
    # two rotations, three roundings each, of pairs of norm r: at most 8 * 2^-24 r
    pair = np.sqrt(x[:, :5, :32] ** 2 + x[:, :5, 32:] ** 2)
    assert np.all(np.abs(_f32(back) - x[:, :5]) <= 8 * 2.0 ** -24 * np.concatenate((pair, pair), -1))
    S.rope([qkv[:, :5]], pos, table, outs=[qkv[:, :5]])
    assert _same(_f32(qkv[:, :5]), want[:, :5]) and _same(_f32(qkv[:, 5:]), x[:, 5:])
    off = torch.empty(T * D + 1, device="cuda")[1:].view(T, 1, D)      # one element off alignment
    off.copy_(dev(x[:, :1]))
    assert _same(_f32(S.rope([off], pos, table)[0]), want[:, :1])


def test_rope_gradient_against_differences():
    """The rotation is linear, so a difference along v equals rope(v): <dy, rope(v)> = <rope^-1(dy), v>."""
    g = rng(6)
    table = dev(R.rope_table(S.rope_frequencies(48)[0], 64, 1.3))
    pos = dev(g.integers(0, 64, 11).astype(np.int32))
    v, vt = _t(g, (11, 3, 64), "f32")
    dy, dyt = _t(g, (11, 3, 64), "f32")
    y = _f32(S.rope([vt], pos, table)[0]).astype(np.float64)
    dx = _f32(S.rope([dyt], pos, table, inverse=True)[0]).astype(np.float64)
    assert abs((dy * y).sum() - (dx * v).sum()) <= 1e-6 * np.abs(dy * y).sum()


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("D,Rt,Hq,Hk,ps,xd,inter", [(128, 128, 20, 5, 16, "f32", False),
                                                    (80, 32, 4, 1, 7, "bf16", True),
                                                    (64, 64, 3, 3, 1, "f32", True),
                                                    (256, 128, 4, 2, 64, "bf16", False),
                                                    (96, 48, 25, 25, 24, "f32", False),
                                                    (80, 20, 4, 2, 16, "bf16", False),   # pairs that
                                                    (64, 22, 3, 1, 16, "f32", False),    # no vector holds
                                                    (48, 30, 2, 2, 8, "f32", True),
                                                    (16, 2, 1, 1, 4, "bf16", False)])
@pytest.mark.parametrize("T", [1, 13, 260])
def test_append(kv, D, Rt, Hq, Hk, ps, xd, inter, T):
    import torch
    g = rng(D + T)
    seqs, per = 6, 12
    pages = seqs * per + 2
    P = per * ps + 5
    table = R.rope_table(S.rope_frequencies(Rt)[0], P - 3)
    blocks = g.permutation(pages)[:seqs * per].reshape(seqs, per).astype(np.int32)
    blocks[2, 0], blocks[3, 0] = -1, pages           # no page; a page that is not the cache's
    slots = [(s, p) for s in range(seqs) for p in range(P)]
    pick = g.permutation(len(slots))[:T] if T <= len(slots) else np.arange(len(slots))
    T = len(pick)
    seq = np.array([slots[i][0] for i in pick], np.int32)
    pos = np.array([slots[i][1] for i in pick], np.int32)
    if T > 4:
        pos[1], seq[2], seq[3] = -1, -1, seqs
    q, qt = _t(g, (T, Hq, D), xd)
    k, kt = _t(g, (T, Hk, D), xd)
    v, vt = _t(g, (T, Hk, D), xd)
    k[0] = 0
    kt[0] = 0
    shape = (pages, Hk, ps, D)
    if kv == "bf16":
        _, kc = _t(g, shape, "bf16")
        _, vc = _t(g, shape, "bf16")
        ks = vs = None
    else:
        kc, vc = (dev(g.integers(-127, 128, shape).astype(np.int8)) for _ in range(2))
        ks, vs = (dev(g.random(shape[:3]).astype(np.float32)) for _ in range(2))
    ref = [_f32(c) for c in (kc, vc)] + ([host(ks).copy(), host(vs).copy()] if kv == "i8" else [])
    print(kv, D, Rt, Hq, Hk, ps, T, flush=True)
    out = S.rope_append(qt, kt, vt, dev(pos), dev(table), kc, vc, dev(blocks), dev(seq), ks, vs, inter,
                        dtype=torch.float32)
    assert _same(_f32(out), R.rope(q, pos, table, inter))
    kr = R.rope(k, pos, table, inter)
    for t in range(T):
        s, p = seq[t], pos[t]
        if not (0 <= s < seqs and 0 <= p < len(table) and p // ps < per):
            continue
        pg, off = blocks[s, p // ps], p % ps
        if not 0 <= pg < pages:
            continue
        for i, x in enumerate((kr[t], v[t])):
            if kv == "bf16":
                ref[i][pg, :, off] = R.bf16_round(x)
            else:
                a, sc = O.act_quant(x)
                ref[i][pg, :, off], ref[2 + i][pg, :, off] = a, sc
    for got, want in zip((kc, vc, ks, vs), ref):
        assert _same(_f32(got), want)


def test_append_decode_step_without_sequence_list_and_token_major_cache():
    """seq None: token t is sequence t; a cache stored [pages][page][heads][D] is a transposed view."""
    g = rng(9)
    B, Hq, Hk, D, ps = 5, 8, 2, 64, 4
    table = R.rope_table(S.rope_frequencies(D)[0], 40)
    blocks = np.arange(B * 10, dtype=np.int32).reshape(B, 10)[::-1].copy()
    pos = g.integers(0, 40, B).astype(np.int32)
    store = [dev(np.zeros((B * 10, ps, Hk, D), np.float32)).bfloat16() for _ in range(2)]
    kc, vc = (c.transpose(1, 2) for c in store)
    x, qkv = _t(g, (B, Hq + 2 * Hk, D), "bf16")
    S.rope_append(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], dev(pos), dev(table), kc, vc,
                  dev(blocks))
    kr = R.bf16_round(R.rope(x[:, Hq:Hq + Hk], pos, table))
    got_k, got_v = (_f32(c) for c in store)
    for b in range(B):
        pg, off = blocks[b, pos[b] // ps], pos[b] % ps
        assert _same(got_k[pg, off], kr[b]) and _same(got_v[pg, off], x[b, Hq + Hk:])
        got_k[pg, off] = 0
        got_v[pg, off] = 0
    assert not got_k.any() and not got_v.any()


@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_append_from_rows_of_any_alignment(xd):
    """Queries, keys and values one element off alignment, with odd strides; queries in place."""
    import torch
    g = rng(31)
    T, Hq, Hk, D, ps = 7, 4, 2, 32, 8
    W = Hq * D + 2 * Hk * D + 3
    table = R.rope_table(S.rope_frequencies(16)[0], 30)
    x, _ = _t(g, (T, W), xd)
    buf = torch.empty(T * W + 1, dtype=torch.float32 if xd == "f32" else torch.bfloat16, device="cuda")[1:]
    buf.copy_(dev(x.reshape(-1)))
    rows = buf.view(T, W)
    cut = lambda a, h: rows[:, a:a + h * D].unflatten(1, (h, D))
    q, k, v = cut(1, Hq), cut(1 + Hq * D, Hk), cut(2 + (Hq + Hk) * D, Hk)
    pos = g.integers(0, 30, T).astype(np.int32)
    blocks = np.arange(T * 4, dtype=np.int32).reshape(T, 4)
    kc, vc = (torch.zeros(T * 4, Hk, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want_q = R.rope(x[:, 1:1 + Hq * D].reshape(T, Hq, D), pos, table)
    want_k = R.bf16_round(R.rope(x[:, 1 + Hq * D:1 + (Hq + Hk) * D].reshape(T, Hk, D), pos, table))
    want_v = R.bf16_round(x[:, 2 + (Hq + Hk) * D:2 + (Hq + 2 * Hk) * D].reshape(T, Hk, D))
    out = S.rope_append(q, k, v, dev(pos), dev(table), kc, vc, dev(blocks), out=q)
    assert _same(_f32(out), want_q if xd == "f32" else R.bf16_round(want_q))
    for t in range(T):
        pg, off = blocks[t, pos[t] // ps], pos[t] % ps
        assert _same(_f32(kc)[pg, :, off], want_k[t]) and _same(_f32(vc)[pg, :, off], want_v[t])
