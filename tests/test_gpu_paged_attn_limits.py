"""Decode attention at the limits of its arithmetic, its workspace and its launch, against the formula
in 64 bits.  u = 2^-24 is half a unit in the last place of a 24-bit float at 1."""
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


def _query(x, qd):
    return _bf16(x) if qd == "bf16" else (np.asarray(x, np.float32), dev(np.asarray(x, np.float32)))


def _terms(p):
    """The leading two bf16 terms of fp32 values."""
    hi = R.bf16_round(p)
    return hi, R.bf16_round(p - hi)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("qd", ["bf16", "f32"])
def test_weights_enter_the_product_with_24_bits(kv, qd):
    """Three keys with weights 1, 1 and p, values -hi, -mid and 1, where hi + mid are the two leading bf16
    terms of p: what is left, under 64 u p, is lost if the weight enters the product as two terms.

    With scores 0, 0, -x, 0 < x <= 1: x carries three roundings (u x each in p's exponent, p x <= 0.37),
    the exponential 2 u, the sum of six products at most 6 u; divided by 2 + p >= 2.  The bf16 output rounds
    a result below 32 u by 2^-9 of it.
    """
    B, Hq, D, ps = 64, 3, 16, 4
    g = rng(41)
    x = (g.integers(1, 128, B) / 128).astype(np.float32)          # bf16 holds it
    kc, vc = np.zeros((B, 1, ps, D), np.float32), np.zeros((B, 1, ps, D), np.float32)
    ks = vs = kst = vst = None
    if kv == "bf16":
        p = np.exp(-x.astype(np.float64)).astype(np.float32)
        hi, mid = _terms(p)
        kc[:, 0, 2, 0] = -x
        for j, v in enumerate((-hi, -mid, np.ones(B))):
            vc[:, 0, j] = np.asarray(v, np.float32)[:, None]
        kt, vt = _bf16(kc)[1], _bf16(vc)[1]
    else:                                     # the same keys and values as a whole number and a scale
        ks, vs = np.ones((B, 1, ps), np.float32), np.ones((B, 1, ps), np.float32)
        ks[:, 0, 2] = x / np.float32(100)
        p = np.exp(-100 * ks[:, 0, 2].astype(np.float64)).astype(np.float32)
        hi, mid = _terms(p)
        kc[:, 0, 2, 0] = -100
        vs[:, 0, 0], vs[:, 0, 1] = hi, np.abs(mid)
        vc[:, 0, 0] = -1
        vc[:, 0, 1] = -np.sign(mid)[:, None]
        vc[:, 0, 2] = 1
        kc, vc = kc.astype(np.int8), vc.astype(np.int8)
        kt, vt, kst, vst = (dev(a) for a in (kc, vc, ks, vs))
    q = np.zeros((B, Hq, D), np.float32)
    q[..., 0] = 1
    q, qt = _query(q, qd)
    blocks, lens = np.arange(B, dtype=np.int32)[:, None], np.full(B, 3, np.int32)
    want, _, _, _ = R.paged_attn(q, kc, vc, blocks, lens, 1.0, 0, ks, vs)
    assert np.abs(want).max() > 10 * U        # a loss of the third term would be seen
    out = S.PagedAttn(B, Hq, 1, D, ps, 3)(qt, kt, vt, dev(blocks), dev(lens), 1.0, kst, vst)
    bound = (3 * 0.37 + 2 + 6) / 2 * U + 2.0 ** -9 * np.abs(want)
    assert np.all(np.abs(_f32(out) - want) <= bound), np.max(np.abs(_f32(out) - want)) / U


def test_one_workspace_for_several_plans():
    """Launches of different plans take turns on one workspace that was zeroed once."""
    import torch
    g = rng(43)
    Hq, Hk, D, ps, per = 16, 8, 64, 16, 40
    pages = 64 * per
    kt, vt = (_bf16(g.standard_normal((pages, Hk, ps, D)))[1] for _ in range(2))
    blocks = dev(g.permutation(pages).reshape(64, per).astype(np.int32))
    lens = dev(g.integers(1, per * ps + 1, 64).astype(np.int32))
    q = dev(g.standard_normal((64, Hq, D)).astype(np.float32))
    sizes = [(64, 16), (1, 16), (64, 8), (7, 16), (3, 8)]
    plans = [S.PagedAttn(B, hq, Hk, D, ps, per * ps) for B, hq in sizes]
    call = lambda p, B, hq: p(q[:B, :hq], kt, vt, blocks[:B], lens[:B], want_lse=True)
    alone = [[t.clone() for t in call(p, *s)] for p, s in zip(plans, sizes)]
    shared = torch.zeros(max(p.plan.ws_bytes for p in plans), dtype=torch.uint8, device="cuda")
    for p in plans:
        p.ws = shared
    for i in [0, 1, 0, 2, 3, 0, 4, 2, 1, 3, 0, 4]:
        B, hq = sizes[i]
        out, lse = torch.full((B, hq, D), 7.0, device="cuda"), torch.full((B, hq), 7.0, device="cuda")
        plans[i](q[:B, :hq], kt, vt, blocks[:B], lens[:B], out=out, lse=lse)
        assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1]), i


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("qd", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,n,top", [(4, 1, 1), (4, 70, 70), (16, 700, 700), (40, 300, 1 << 20)])
def test_infinite_values_reach_their_elements_as_in_the_formula(kv, qd, Hq, n, top):
    """A live infinite value makes its element of the output infinite, infinities of both signs (int8: an
    infinite scale of a zero) make it NaN, and every other element is what it is without them."""
    g = rng(47 + n)
    B, D, ps = 3, 32, 16
    per = -(-n // ps)
    pages = B * per
    q, qt = _query(g.standard_normal((B, Hq, D)), qd)
    k = g.standard_normal((pages, 1, ps, D))
    ks = vs = kst = vst = None
    blocks, lens = np.arange(pages, dtype=np.int32).reshape(B, per), np.full(B, n, np.int32)
    at = [(t // ps, t % ps) for t in sorted({0, n // 2, n - 1})]      # of sequence 0
    if kv == "bf16":
        k, kt = _bf16(k)
        v, vt = _bf16(g.standard_normal(k.shape))
        clean, cleant = v, vt
        v = v.copy()
        for i, (p, o) in enumerate(at):
            v[p, 0, o, 3 + i], v[p, 0, o, 9 + i] = np.inf, -np.inf
        p, o = at[-1]
        v[p, 0, o, 20], v[at[0][0], 0, at[0][1], 20] = -np.inf, np.inf
        vt = _bf16(v)[1]
        clean_vs = cleanst = None
    else:
        k, v = (g.integers(-127, 128, k.shape).astype(np.int8) for _ in range(2))
        p, o = at[0]
        v[p, 0, o, :4] = 0, 1, -1, 127
        ks, vs = ((0.01 + 0.01 * g.random(k.shape[:3])).astype(np.float32) for _ in range(2))
        clean, clean_vs = v, vs
        vs = vs.copy()
        vs[p, 0, o] = np.inf
        kt, vt, kst, vst, cleanst = (dev(a) for a in (k, v, ks, vs, clean_vs))
        cleant = vt
    plan = S.PagedAttn(B, Hq, 1, D, ps, top)
    with np.errstate(invalid="ignore"):
        want, wl, _, _ = R.paged_attn(q, k, v, blocks, lens, D ** -0.5, 0, ks, vs)
    call = lambda vt, vst: [host(t.float()) for t in plan(qt, kt, vt, dev(blocks), dev(lens), k_scale=kst,
                                                           v_scale=vst, want_lse=True)]
    got, lse = call(vt, vst)
    base, base_lse = call(cleant, cleanst)
    odd = ~np.isfinite(want)
    assert odd[0].any() and not odd[1:].any()
    assert np.array_equal(got[odd], want[odd], equal_nan=True)
    assert np.array_equal(got[~odd], base[~odd]) and np.array_equal(lse, base_lse)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_queries_enter_the_product_with_24_bits(kv):
    """fp32 queries (a, hi, mid) against keys 2^14 (1, -1, -1), where hi + mid are the two leading bf16
    terms of a: the score is 2^14 of what is left of a, exact in every step but the last roundings, and the
    score of a query held as two terms would be 0.  One key, so lse is the score."""
    B, Hq, D, ps = 8, 16, 16, 1
    g = rng(53)
    a = (1 + g.random((B, Hq))).astype(np.float32)
    hi, mid = _terms(a)
    q = np.zeros((B, Hq, D), np.float32)
    q[..., 0], q[..., 1], q[..., 2] = a, hi, mid
    c = 2.0 ** 14
    kc = np.zeros((B, 1, ps, D), np.float32)
    kc[..., 0], kc[..., 1:3] = 1, -1
    ks = kst = vst = None
    if kv == "bf16":
        kt, vt = _bf16(kc * c)[1], _bf16(np.ones_like(kc))[1]
    else:
        kt, vt = dev(kc.astype(np.int8)), dev(np.ones(kc.shape, np.int8))
        kst, vst = dev(np.full((B, 1, ps), c, np.float32)), dev(np.ones((B, 1, ps), np.float32))
    blocks, lens = np.arange(B, dtype=np.int32)[:, None], np.ones(B, np.int32)
    want = c * (a.astype(np.float64) - hi - mid)
    assert np.abs(want).max() > 0.02
    out, lse = S.PagedAttn(B, Hq, 1, D, ps, 1)(dev(q), kt, vt, dev(blocks), dev(lens), 1.0, kst, vst, want_lse=True)
    # sums of mid and lo parts: three of at most 2^14 * 2^-8, rounded; then three roundings to and from log2
    assert np.all(np.abs(host(lse) - want) <= 3 * U * 2.0 ** 6 + 6 * U * np.abs(want))
    assert np.array_equal(_f32(out), np.ones_like(q))


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_queries_at_the_end_of_the_fp32_range(kv):
    """Queries that a rounding to bf16 would carry to infinity, against keys that bring the score back:
    one key of score q k and one of score 0."""
    B, D, ps = 1, 16, 4
    big = np.array([3.4028235e38, -3.4028235e38, 3.399e38, 3.39e38, -3.3962e38, 1.0], np.float32)
    Hq = len(big)
    q = np.zeros((B, Hq, D), np.float32)
    q[0, :, 5] = big
    tiny = 2.0 ** -125
    kc, vc = np.zeros((1, 1, ps, D), np.float32), np.zeros((1, 1, ps, D), np.float32)
    ks = vs = kst = vst = None
    if kv == "bf16":
        kc[0, 0, 1, 5] = tiny
        vc[0, 0, 1] = 1
        kt, vt = _bf16(kc)[1], _bf16(vc)[1]
        scale = 0.5
    else:
        kc[0, 0, 1, 5] = vc[0, 0, 1, 0] = 1
        ks, vs = (np.full((1, 1, ps), s, np.float32) for s in (tiny, 1.0))
        kc, vc = kc.astype(np.int8), vc.astype(np.int8)
        kt, vt, kst, vst = (dev(a) for a in (kc, vc, ks, vs))
        scale = 0.5
    blocks, lens = np.zeros((1, 1), np.int32), np.full(1, 2, np.int32)
    want, wl, mag, smag = R.paged_attn(q, kc, vc, blocks, lens, scale, 0, ks, vs)
    out, lse = S.PagedAttn(B, Hq, 1, D, ps, 2)(dev(q), kt, vt, dev(blocks), dev(lens), scale, kst, vst, want_lse=True)
    e = (8 * U * smag + 8 * U)[..., None]     # a score's few roundings, the exponential's and the sums'
    assert np.all(np.abs(_f32(out) - want) <= 2 * e * mag + 1e-30)
    assert np.all(np.abs(host(lse) - wl) <= e[..., 0] + 4 * U * np.abs(wl))


def test_values_at_the_end_of_the_fp32_range():
    """An int8 value times a scale that a rounding to bf16 would carry to infinity."""
    B, Hq, D, ps = 1, 2, 16, 4
    vs = np.full((1, 1, ps), 3.4028235e38, np.float32)
    kt, vt = dev(np.zeros((1, 1, ps, D), np.int8)), dev(np.ones((1, 1, ps, D), np.int8))
    out = S.PagedAttn(B, Hq, 1, D, ps, 1)(dev(np.ones((B, Hq, D), np.float32)), kt, vt,
                                          dev(np.zeros((1, 1), np.int32)), dev(np.ones(1, np.int32)),
                                          k_scale=dev(np.ones((1, 1, ps), np.float32)), v_scale=dev(vs))
    assert np.array_equal(_f32(out), np.full((B, Hq, D), vs[0, 0, 0]))


def test_a_query_that_is_nan_in_its_last_bits():
    B, Hq, D, ps = 1, 4, 16, 4
    q = np.ones((B, Hq, D), np.float32)
    q[0, 1:, 3].view(np.uint32)[:] = [0x7F800001, 0xFF800001, 0x7FC00000]
    kt, vt = _bf16(np.full((1, 1, ps, D), -1.0))[1], _bf16(np.ones((1, 1, ps, D)))[1]
    out, lse = S.PagedAttn(B, Hq, 1, D, ps, 3)(dev(q), kt, vt, dev(np.zeros((1, 1), np.int32)),
                                               dev(np.full(1, 3, np.int32)), want_lse=True)
    assert np.array_equal(_f32(out)[0, 0], np.ones(D)) and np.isfinite(host(lse)[0, 0])
    assert np.all(np.isnan(_f32(out)[0, 1:])) and np.all(np.isnan(host(lse)[0, 1:]))


def _repeating(g, Hk, ps, D, kv, own):
    """A cache of `own` pages of random rows, for block tables that name its pages again and again."""
    shape = (own, Hk, ps, D)
    if kv == "bf16":
        (k, kt), (v, vt) = _bf16(g.standard_normal(shape)), _bf16(g.standard_normal(shape))
        return k, v, None, None, kt, vt, None, None
    k, v = (g.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
    ks, vs = ((0.005 + 0.02 * g.random(shape[:3])).astype(np.float32) for _ in range(2))
    return (k, v, ks, vs) + tuple(dev(a) for a in (k, v, ks, vs))


def _close(out, lse, q, c, blocks, lens, window=0):
    """Within a bound counted from the arithmetic with fp32 queries: scores of D products ((D + 6) u of the
    absolute ones), 4 u an exponential, n + 64 sums of weights; and near the plain form's error on the
    whole (32-bit operations give 2 to 8e-7)."""
    D = q.shape[2]
    want, wl, mag, smag = R.paged_attn(q, c[0], c[1], blocks, lens, D ** -0.5, window, c[2], c[3])
    e = ((D + 6) * U * smag + 4 * U + (np.max(lens) + 64) * U)[..., None]
    got, gl = _f32(out), host(lse)
    assert np.all(np.abs(got - want) <= 2 * e * mag + 4 * U * np.abs(want) + 1e-30)
    assert np.linalg.norm(got - want) <= 1e-6 * np.linalg.norm(want)
    dead = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), dead)
    assert np.all(np.abs(gl[~dead] - wl[~dead]) <= e[..., 0][~dead] + 4 * U * np.abs(wl[~dead]))


def test_strides_of_axes_of_one():
    """The stride of an axis of one element is never a step, whatever it is: one sequence cut out of rows
    of odd length, a cache of one page, one head, or one slot per page."""
    g = rng(61)
    D, ps = 32, 4
    x = g.standard_normal((1, 4 * D)).astype(np.float32)
    q, qt = x.reshape(1, 4, D), dev(x).as_strided((1, 4, D), (4 * D + 3, D, 1))
    wide = dev(x).as_strided((1, 1, D), (1, 3, 1))
    for shape, fake in (((1, 2, ps, D), 0), ((3, 1, ps, D), 1), ((6, 2, 1, D), 2), ((1, 1, 1, D), None)):
        pages, Hk, slots, _ = shape
        for kv in ("bf16", "i8"):
            c = _repeating(g, Hk, slots, D, kv, pages)
            strides = list(c[4].stride())
            for a in range(3):
                if a == fake or (fake is None and shape[a] == 1):
                    strides[a] = 3 + 2 * a
            kt, vt = c[4].as_strided(shape, strides), c[5]
            if kv == "bf16":                  # both alike
                vt = vt.as_strided(shape, strides)
            blocks = np.arange(pages, dtype=np.int32)[None]
            lens = np.full(1, pages * slots, np.int32)
            for a, at in ((q, qt), (q[:, :1], wide)):
                if a.shape[1] % Hk:
                    continue
                out, lse = S.PagedAttn(1, a.shape[1], Hk, D, slots, 8)(
                    at, kt, vt, dev(blocks), dev(lens), k_scale=c[6], v_scale=c[7], want_lse=True)
                _close(out, lse, a, c, blocks, lens)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("Hq,Hk,D,n,runs,rows", [
    (16, 1, 64, 131072, 145, 16),    # the runs' weights fill LDS several times over
    (16, 1, 128, 131072, 401, 16),
    (16, 1, 256, 60000, 65, 16),     # more runs than a thread holds the maxima of
    (5, 1, 48, 50000, 65, 16),
    (20, 1, 64, 131072, 333, 32),    # two query tiles
    (24, 1, 128, 70000, 33, 32)])
def test_joins_of_many_runs(kv, Hq, Hk, D, n, runs, rows):
    g = rng(D + n)
    ps, own, B = 64, 37, 1
    if rows == 32:                            # a batch whose bound asks for two tiles, one sequence alone is long
        B = 16
    per = -(-n // ps)
    c = _repeating(g, Hk, ps, D, kv, own)
    blocks = g.integers(0, own, (B, per)).astype(np.int32)
    lens = g.integers(0, 40, B).astype(np.int32)
    lens[B // 2] = n
    q = g.standard_normal((B, Hq, D)).astype(np.float32)
    plan = S.PagedAttn(B, Hq, Hk, D, ps, n)
    assert plan.plan.q_rows == rows and plan.plan.blocks > runs
    print(kv, Hq, Hk, D, n, plan.plan.blocks, flush=True)
    for _ in range(2):
        out, lse = plan(dev(q), c[4], c[5], dev(blocks), dev(lens), k_scale=c[6], v_scale=c[7], want_lse=True)
        _close(out, lse, q, c, blocks, lens)


@pytest.mark.parametrize("B", [63, 64, 65, 128, 129, 200, 1000])
@pytest.mark.parametrize("kv,Hq,Hk", [("bf16", 2, 1), ("i8", 6, 3)])
def test_batches_past_64_sequences(B, kv, Hq, Hk):
    """The search for a block's first sequence runs 64 sequences at a time: ragged batches with empty
    sequences, and none but empty ones, at its edges."""
    g = rng(B)
    D, ps, top, own = 32, 8, 500, 11
    per = -(-top // ps)
    c = _repeating(g, Hk, ps, D, kv, own)
    blocks = g.integers(0, own, (B, per)).astype(np.int32)
    lens = g.integers(0, top + 1, B).astype(np.int32)
    for i in (0, 62, 63, 64, 65, 127, 128, B - 1):
        if i < B:
            lens[i] = 0
    q = g.standard_normal((B, Hq, D)).astype(np.float32)
    plan = S.PagedAttn(B, Hq, Hk, D, ps, top)
    one = np.where(np.arange(B) == B - 1, top, 0).astype(np.int32)
    late = np.where(np.arange(B) >= 64, lens, 0).astype(np.int32)
    for n in (lens, one, late, lens, np.zeros_like(lens)):
        out, lse = plan(dev(q), c[4], c[5], dev(blocks), dev(n), k_scale=c[6], v_scale=c[7], want_lse=True)
        _close(out, lse, q, c, blocks, n)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("B,Hq,Hk,D,ps,top", [(1, 20, 5, 128, 16, 700), (3, 8, 8, 64, 1, 130), (5, 4, 1, 80, 24, 300),
                                              (2, 40, 2, 128, 8, 77), (7, 2, 1, 256, 64, 1500),
                                              (2, 33, 1, 96, 16, 520), (1, 1, 1, 16, 3, 40),
                                              (4, 16, 1, 48, 256, 5000), (2, 6, 2, 208, 5, 600)])
def test_fp32_queries_are_as_good_as_32_bit_operations(kv, B, Hq, Hk, D, ps, top):
    g = rng(B * 31 + D + top)
    per = -(-top // ps) + 1
    c = _repeating(g, Hk, ps, D, kv, B * per)
    blocks = g.permutation(B * per).reshape(B, per).astype(np.int32)
    lens = g.integers(1, top + 1, B).astype(np.int32)
    lens[0] = top
    q = g.standard_normal((B, Hq, D)).astype(np.float32)
    out, lse = S.PagedAttn(B, Hq, Hk, D, ps, top)(dev(q), c[4], c[5], dev(blocks), dev(lens), k_scale=c[6],
                                                  v_scale=c[7], want_lse=True)
    _close(out, lse, q, c, blocks, lens)
