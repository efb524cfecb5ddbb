"""Decode attention over a paged cache against the formula in 64 bits.

The bound per output element is counted from the arithmetic: a score is a sum of D exact products in
fp32, off by at most (D + 4) u sum|q k| (u = 2^-24; three bf16 terms hold an fp32 query exactly), an
exponential is good to 4 u, the two bf16 terms of a probability to 2^-17, the sums over n keys round
at most n + 64 times; a relative error e of every weight moves sum(p v) / sum(p) by at most 2 e of
sum(p |v|) / sum(p).  The output is then rounded to its type.
"""
import numpy as np
import pytest

import oracle.block_ref as R
from parity_util import bf16_dev, dev, host
from synth import rng, to_bf16

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")
U = 2.0 ** -24


def _f32(t):
    return host(t.float())


def _bf16(x):
    v, bits = to_bf16(np.asarray(x, np.float32))
    return v, bf16_dev(bits)


class Cache:
    def __init__(self, g, pages, heads, ps, D, kv, std=1.0):
        shape = (pages, heads, ps, D)
        self.ks = self.vs = self.kst = self.vst = None
        if kv == "bf16":
            self.k, self.kt = _bf16(g.standard_normal(shape) * std)
            self.v, self.vt = _bf16(g.standard_normal(shape))
        else:
            self.k, self.v = (g.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
            self.ks, self.vs = ((0.005 + 0.02 * g.random(shape[:3])).astype(np.float32) for _ in range(2))
            self.kt, self.vt, self.kst, self.vst = (dev(a) for a in (self.k, self.v, self.ks, self.vs))


def _check(out, lse, q, c, blocks, lens, window=0, scale=None, bf16=False, n=None):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    want, wl, mag, smag = R.paged_attn(q, c.k, c.v, blocks, lens, scale, window, c.ks, c.vs)
    n = max(1, int(np.max(lens))) if n is None else n
    e = ((D + 6) * U * smag + 4 * U + 2.0 ** -17 + (n + 64) * U)[..., None]
    tol = 2 * e * mag + (2.0 ** -8 if bf16 else 4 * U) * np.abs(want) + 1e-30
    got = _f32(out)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    if not bf16 and np.linalg.norm(want):     # the bound's worst case does not happen: far closer on the whole
        assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)
    dead = np.isneginf(wl)
    gl = host(lse)
    assert np.array_equal(np.isneginf(gl), dead)
    assert np.all(np.abs(gl[~dead] - wl[~dead]) <= (e[..., 0] + 4 * U * np.abs(np.where(dead, 0, wl)))[~dead])


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("qd", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hk,D,ps,top", [(1, 20, 5, 128, 16, 700), (3, 8, 8, 64, 1, 130),
                                              (5, 4, 1, 80, 24, 300), (2, 40, 2, 128, 8, 77),
                                              (7, 2, 1, 256, 64, 1500), (2, 33, 1, 96, 16, 520),
                                              (1, 1, 1, 16, 3, 40), (4, 16, 1, 48, 256, 5000),
                                              (2, 6, 2, 208, 5, 600)])
def test_attention_within_bound(kv, qd, B, Hq, Hk, D, ps, top):
    g = rng(B * 31 + D + top)
    per = -(-top // ps) + 1
    pages = B * per + 2
    c = Cache(g, pages, Hk, ps, D, kv)
    blocks = g.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
    lens = g.integers(0, top + 1, B).astype(np.int32)
    lens[0] = top
    if B > 2:
        lens[1], lens[2] = 0, 1
    q, qt = _bf16(g.standard_normal((B, Hq, D))) if qd == "bf16" else (None, None)
    if q is None:
        q = g.standard_normal((B, Hq, D)).astype(np.float32)
        qt = dev(q)
    plan = S.PagedAttn(B, Hq, Hk, D, ps, top)
    print(kv, qd, B, Hq, Hk, D, ps, top, plan.plan.blocks, flush=True)
    for _ in range(2):                       # the workspace is ready again after a call
        out, lse = plan(qt, c.kt, c.vt, dev(blocks), dev(lens), k_scale=c.kst, v_scale=c.vst, want_lse=True)
        assert out.dtype == qt.dtype
        _check(out, lse, q, c, blocks, lens, bf16=qd == "bf16")


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 127, 128, 129, 255, 256, 257, 385, 511, 513])
def test_lengths_around_the_tiles(kv, n):
    """One batch of sequences of n tokens each side of every tile edge, pages of 20 ending inside tiles."""
    g = rng(n)
    ps, Hk, Hq, D = 20, 2, 6, 64
    per = -(-n // ps)
    c = Cache(g, 3 * per, Hk, ps, D, kv)
    blocks = g.permutation(3 * per).reshape(3, per).astype(np.int32)
    lens = np.array([n, max(0, n - 1), n], np.int32)
    q = g.standard_normal((3, Hq, D)).astype(np.float32)
    for top in (n, 1, 4 * n):                # a plan for just this length, a shorter and a longer bound
        plan = S.PagedAttn(3, Hq, Hk, D, ps, top)
        out, lse = plan(dev(q), c.kt, c.vt, dev(blocks), dev(lens), k_scale=c.kst, v_scale=c.vst, want_lse=True)
        _check(out, lse, q, c, blocks, lens)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_masked_slots_may_hold_anything(kv):
    """Holes in the table, lengths past the table, pages that end inside a tile: slots that are not
    live hold NaN and infinities (int8: NaN scales), live results stay within the bound; a sequence
    all of holes is empty."""
    g = rng(77)
    B, Hq, Hk, D, ps, per = 5, 8, 2, 128, 12, 50
    pages = B * per
    c = Cache(g, pages, Hk, ps, D, kv)
    blocks = g.permutation(pages).reshape(B, per).astype(np.int32)
    lens = np.array([590, 601, 1, 10 ** 6, 300], np.int32)
    first = np.argwhere(blocks == 0)[0]       # page 0 belongs to the sequence of holes: all of it is dead
    blocks[tuple(first)], blocks[4, 0] = blocks[4, 0], 0
    dead = np.ones((pages, ps), bool)
    blocks[0, 3], blocks[0, 40], blocks[1, 0], blocks[1, 49] = -1, pages, -7, 2 ** 31 - 1
    blocks[4] = -1
    for b in range(B):
        for t in range(min(int(lens[b]), per * ps)):
            p = blocks[b, t // ps]
            if 0 <= p < pages:
                dead[p, t % ps] = False
    import torch
    sel = dev(np.broadcast_to(dead[:, None], (pages, Hk, ps)).copy())
    odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device="cuda")
    pick = g.integers(0, 4, (pages, Hk, ps))
    pick[0] = 0                               # the first row is what a masked key's load reads
    junk = odd[dev(pick)]
    if kv == "bf16":
        for t in (c.kt, c.vt):
            t[sel] = junk[sel][:, None].to(t.dtype).expand(-1, D)
    else:
        for t in (c.kst, c.vst):
            t[sel] = junk[sel]
    q = g.standard_normal((B, Hq, D)).astype(np.float32)
    for top in (600, 64, 10 ** 6):
        plan = S.PagedAttn(B, Hq, Hk, D, ps, top)
        out, lse = plan(dev(q), c.kt, c.vt, dev(blocks), dev(lens), k_scale=c.kst, v_scale=c.vst, want_lse=True)
        _check(out, lse, q, c, blocks, lens, n=600)
        assert not _f32(out)[4].any() and np.all(np.isneginf(host(lse)[4]))


@pytest.mark.parametrize("window", [1, 31, 200, 5000])
def test_window(window):
    g = rng(window)
    B, Hq, Hk, D, ps, top = 4, 10, 5, 80, 16, 900
    per = -(-top // ps)
    c = Cache(g, B * per, Hk, ps, D, "bf16")
    blocks = np.arange(B * per, dtype=np.int32).reshape(B, per)
    lens = np.array([900, 0, 17, 450], np.int32)
    q = g.standard_normal((B, Hq, D)).astype(np.float32)
    plan = S.PagedAttn(B, Hq, Hk, D, ps, top, window=window)
    out, lse = plan(dev(q), c.kt, c.vt, dev(blocks), dev(lens), want_lse=True, scale=0.3)
    _check(out, lse, q, c, blocks, lens, window, 0.3)


def test_large_scores_and_values_that_are_not_finite():
    """Scores of thousands (a running maximum that keeps rising), weights of type-lowest keys, and live
    NaN or infinite keys, which reach the result as in the formula."""
    import torch
    g = rng(8)
    B, H, D, ps, n = 4, 2, 64, 16, 400
    per = n // ps
    c = Cache(g, B * per, H, ps, D, "bf16", std=1.0)
    blocks = np.arange(B * per, dtype=np.int32).reshape(B, per)
    ramp = np.repeat(np.linspace(1, 60, per), 1).astype(np.float32)
    for b in range(B):                        # later pages have larger keys
        c.k[b * per:(b + 1) * per] = R.bf16_round(c.k[b * per:(b + 1) * per] * ramp[:, None, None, None])
    low = R.bf16_round(np.float32(-3.0e38))
    q = np.abs(g.standard_normal((B, H, D))).astype(np.float32)
    c.k[per, 0, 3] = 0
    c.k[per, 0, 3, 5] = low                   # a score of the type's lowest magnitude: weight 0
    c.kt.copy_(dev(c.k).bfloat16())
    lens = np.full(B, n, np.int32)
    plan = S.PagedAttn(B, H, H, D, ps, n)
    out, lse = plan(dev(q), c.kt, c.vt, dev(blocks), dev(lens), want_lse=True)
    _check(out, lse, q, c, blocks, lens)
    for value, seq in ((float("nan"), 1), (float("inf"), 2)):
        c.kt[seq * per + 2, :, 7] = value
    out, lse = plan(dev(q), c.kt, c.vt, dev(blocks), dev(lens), want_lse=True)
    got = _f32(out)
    assert np.all(np.isfinite(got[[0, 3]])) and np.all(np.isnan(got[[1, 2]])) and np.all(np.isnan(host(lse)[1]))
    c.kt[3 * per:] = -float("inf")            # every weight is zero: an empty row
    out, lse = plan(dev(q), c.kt, c.vt, dev(blocks), dev(lens), want_lse=True)
    assert not _f32(out)[3].any() and np.all(np.isneginf(host(lse)[3]))


def test_strides_and_a_cache_past_32_bit_offsets():
    """Queries as slices of a fused buffer, a token-major cache as a transposed view, and pages beyond
    2^31 elements of a cache allocated larger than is filled."""
    import torch
    g = rng(15)
    B, Hq, Hk, D, ps = 2, 8, 4, 128, 64
    pages = (2 ** 31) // (Hk * ps * D) + 40
    kt, vt = (torch.empty((pages, ps, Hk, D), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
              for _ in range(2))
    blocks = np.array([[pages - 1, 3, pages - 7], [0, pages - 2, 5]], np.int32)
    c = Cache(g, pages=6, heads=Hk, ps=ps, D=D, kv="bf16")
    flat = blocks.ravel()
    for i, p in enumerate(flat):
        kt[p], vt[p] = c.kt[i], c.vt[i]
    lens = np.array([180, 192], np.int32)
    x = g.standard_normal((B, Hq + 2 * Hk, D)).astype(np.float32)
    xt = dev(x)
    plan = S.PagedAttn(B, Hq, Hk, D, ps, 192)
    out, lse = plan(xt[:, :Hq], kt, vt, dev(blocks), dev(lens), want_lse=True)
    _check(out, lse, x[:, :Hq], c, np.arange(6, dtype=np.int32).reshape(2, 3), lens)


def test_order_of_blocks_does_not_matter_and_graph_replays():
    import torch
    g = rng(21)
    B, Hq, Hk, D, ps, n = 6, 8, 2, 128, 16, 3000
    per = -(-n // ps)
    c = Cache(g, B * per, Hk, ps, D, "bf16")
    blocks = dev(g.permutation(B * per).reshape(B, per).astype(np.int32))
    lens = dev(g.integers(1, n + 1, B).astype(np.int32))
    qt = _bf16(g.standard_normal((B, Hq, D)))[1]
    plan = S.PagedAttn(B, Hq, Hk, D, ps, n)
    assert plan.plan.blocks > B * Hk          # the sequences are split
    first, lse = plan(qt, c.kt, c.vt, blocks, lens, want_lse=True)
    for _ in range(5):
        again, l2 = plan(qt, c.kt, c.vt, blocks, lens, want_lse=True)
        assert torch.equal(first, again) and torch.equal(lse, l2)
    out, lo = torch.empty_like(first), torch.empty_like(lse)
    cap, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr, stream=cap):
        plan(qt, c.kt, c.vt, blocks, lens, out=out, lse=lo)
    for _ in range(4):
        out.fill_(7.0)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(lo, lse)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("qd", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hk,D,ps,top", [(3, 17, 1, 128, 16, 1200), (2, 96, 3, 64, 20, 700),
                                              (4, 33, 1, 40, 8, 129), (1, 71, 1, 96, 64, 3000),
                                              (2, 40, 2, 128, 12, 64)])
def test_two_query_tiles_per_block(kv, qd, B, Hq, Hk, D, ps, top):
    """More than 16 query heads on a key head under a bound of lengths that calls for one reading of the
    keys by 32 of them: within the bound, dead slots may hold anything, and a batch split at its own,
    short bound (one query tile per block) agrees."""
    D = -(-D // 16) * 16 if kv == "i8" else D   # rows of 16 bytes
    g = rng(B * 17 + Hq + top)
    per = -(-top // ps) + 1
    pages = B * per + 1                        # page 0 is masked from the start
    c = Cache(g, pages, Hk, ps, D, kv)
    blocks = 1 + g.permutation(pages - 1)[:B * per].reshape(B, per).astype(np.int32)
    lens = g.integers(0, top + 1, B).astype(np.int32)
    lens[0] = top
    blocks[0, 0] = -1                          # a hole: its keys are dead as well
    dead = np.ones((pages, ps), bool)
    for b in range(B):
        for t in range(int(lens[b])):
            if blocks[b, t // ps] >= 0:
                dead[blocks[b, t // ps], t % ps] = False
    sel = dev(np.broadcast_to(dead[:, None], (pages, Hk, ps)).copy())
    for t in ((c.kt, c.vt) if kv == "bf16" else (c.kst, c.vst)):
        t[sel] = float("nan")
    if qd == "bf16":
        q, qt = _bf16(g.standard_normal((B, Hq, D)))
    else:
        q = g.standard_normal((B, Hq, D)).astype(np.float32)
        qt = dev(q)
    bound = 128 * (1 << 16) // (B * Hk) ** 2 + 1024 * 128
    wide, near = S.PagedAttn(B, Hq, Hk, D, ps, bound), S.PagedAttn(B, Hq, Hk, D, ps, top)
    assert (wide.plan.q_rows, near.plan.q_rows) == (32, 16)
    print(kv, qd, B, Hq, Hk, D, ps, top, wide.plan.blocks, flush=True)
    for plan in (wide, near, wide):
        out, lse = plan(qt, c.kt, c.vt, dev(blocks), dev(lens), k_scale=c.kst, v_scale=c.vst, want_lse=True)
        _check(out, lse, q, c, blocks, lens, bf16=qd == "bf16")
