"""Tokens drawn from logits, equal to those of the token-by-token restatement, and their log probabilities.

The log probability's bound: a term of the sum is exp2 (one ulp, 2^-23) of a difference and a product rounded
to fp32 (2^-24 each of an exponent d): relative error of the sum at most 2^-23 (1 + sum p_i |d_i|) to first order,
doubled here for what is behind it; the result is rounded once.
"""
import numpy as np
import pytest

import oracle.step_ref as R
from parity_util import dev, host
from synth import rng

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")

INF, NAN = np.inf, np.nan


def _upload(x, xd):
    t = dev(np.asarray(x, np.float32))
    if xd == "bf16":
        t = t.bfloat16()
        x = host(t.float())
    return t, np.asarray(x, np.float32)


def _check(x, u, temperature=None, k=None, p=None, min_p=None, xd="f32", t=None):
    B, V = np.shape(x)
    if t is None:
        t, x = _upload(x, xd)
    per = lambda v, d: None if v is None else np.broadcast_to(np.asarray(v, d), (B,)).copy()  # noqa: E731
    u, temperature, k, p, min_p = per(u, np.float64), per(temperature, np.float32), per(k, np.int32), per(
        p, np.float32), per(min_p, np.float32)
    up = lambda v: None if v is None else dev(v)  # noqa: E731
    token, logprob = S.sample(t, dev(u), up(temperature), up(k), up(p), up(min_p), want_logprob=True)
    token, logprob = host(token), host(logprob).astype(np.float64)
    for b in range(B):
        at = lambda v, none: none if v is None else v[b]  # noqa: B023, E731
        want, lp, d = R.sample_row(x[b], u[b], at(temperature, 1.0), at(k, 0), at(p, 1.0), at(min_p, 0.0))
        assert token[b] == want, (b, V, u[b], at(temperature, 1.0), at(k, 0), at(p, 1.0), at(min_p, 0.0))
        if np.isfinite(lp):
            assert abs(logprob[b] - lp) <= 2.0 ** -22 * (1 + d) + 2.0 ** -24 * abs(lp), (logprob[b], lp)
        else:
            assert logprob[b] == lp
    return token


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.7), dict(k=1), dict(k=5), dict(k=300, temperature=1.3),
            dict(p=0.9), dict(p=0.5, temperature=2.0), dict(min_p=0.05), dict(k=40, p=0.95), dict(k=2000, p=0.3),
            dict(k=50, p=0.9, min_p=0.1, temperature=0.8), dict(p=0.0), dict(min_p=2.0), dict(p=0.999, min_p=1e-7)]


@pytest.mark.parametrize("V", [1, 2, 7, 8, 63, 64, 65, 1000, 2047, 2048, 2049, 4097, 10007])
@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_settings(V, xd):
    g = rng(V)
    for kw in SETTINGS:
        x = g.standard_normal((3, V)) * g.choice([0.3, 2.5, 8.0])
        _check(x, g.random(3), xd=xd, **kw)


@pytest.mark.parametrize("V,B", [(50000, 2), (131072, 2), (262144, 1), (33001, 5)])
@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_large_vocabularies(V, B, xd):
    g = rng(V + 1)
    for kw in SETTINGS:
        _check(g.standard_normal((B, V)) * 2.5, g.random(B), xd=xd, **kw)


def test_flat_rows_keep_many_tokens():
    """Kept sets of tens of thousands of tokens: every question about the order takes a pass of its own."""
    g = rng(6)
    x = g.standard_normal((2, 100000)) * 0.5
    for kw in [dict(k=60000), dict(p=0.7), dict(k=70000, p=0.9), dict(k=30000, p=0.2), dict(min_p=0.2, p=0.99)]:
        _check(x, g.random(2), **kw)


@pytest.mark.parametrize("B", [1, 3, 17, 200, 1100])
def test_rows_with_settings_of_their_own(B):
    g = rng(B)
    V = 3001
    x = g.standard_normal((B, V)) * 3
    x[g.random((B, V)) < 0.3] = -INF
    _check(x, g.random(B), g.choice([0, 0.5, 1, 2, -1, NAN], B), g.choice([0, -3, 1, 30, V, 2 ** 31 - 1], B),
           g.choice([1, 0.9, 0.2, 1.5, -1, NAN], B), g.choice([0, 0.1, -1, NAN, 0.01], B))


@pytest.mark.parametrize("B,V", [(130, 40011), (3, 300007), (129, 16390)])
def test_rows_in_parts_of_several_turns(B, V):
    """A block's part of a row is more than it counts at a time, and its last turn is not whole."""
    g = rng(V)
    x = g.standard_normal((B, V)) * 2.5
    x[g.random((B, V)) < 0.05] = -INF
    x[1] = np.sort(x[1])                       # all of what weighs most in one part
    _check(x, g.random(B), g.choice([1, 0.7, 1.2, 0], B), g.choice([0, 20, 700, V // 2], B), g.choice([1, 0.9, 0.98], B),
           g.choice([0, 0.02], B))


@pytest.mark.parametrize("V,std", [(81063, 1.0), (262143, 1.0), (50000, 0.3), (131072, 5.0)])
def test_bf16_rows_hold_many_equal_logits(V, std):
    """Hundreds of tokens with the logit in question, not next to each other."""
    g = rng(V)
    x = g.standard_normal((3, V)) * std
    for kw in [dict(temperature=1.5), dict(p=0.9), dict(k=V // 3), dict(k=V // 2, p=0.97), dict(min_p=0.001, p=0.99)]:
        for _ in range(2):
            _check(x, g.random(3), xd="bf16", **kw)


def test_greedy_rows_in_parts_of_several_turns():
    g = rng(3)
    x = g.standard_normal((130, 40011)) * 3
    _check(x, g.random(130), 0.0)


@pytest.mark.parametrize("V", [5, 100, 4096, 4097, 20000, 70000])
@pytest.mark.parametrize("kw", [dict(), dict(k=3), dict(p=0.5), dict(min_p=0.5), dict(temperature=0.0), dict(k=4500, p=0.6)])
def test_equal_logits(V, kw):
    """Ties go by index; more of them than a row's block sorts are counted."""
    u = np.array([0.0, 0.3, 0.999999, 1 - 2.0 ** -53])
    _check(np.full((4, V), 1.25), u, **kw)


def test_many_equal_logits_below_others():
    g = rng(9)
    V = 30000
    x = np.full((6, V), -1.0)
    x[:, g.permutation(V)[:500]] = g.standard_normal((6, 500))
    x[3:, ::2] = -1.0 - 2.0 ** -23           # beside them by an ulp
    for kw in [dict(), dict(k=5000), dict(k=20001, p=0.95), dict(p=0.8), dict(min_p=0.1)]:
        _check(x, g.random(6), **kw)


def test_close_logits_in_a_wide_range():
    """Thousands of different logits in one bin, because others are far below."""
    g = rng(10)
    V = 40000
    x = 3.0 + g.standard_normal((4, V)) * 1e-4
    x[:, :10] = np.finfo(np.float32).min
    x[2:, 10:9000] = -20.0
    for kw in [dict(), dict(k=7000), dict(p=0.3), dict(k=25000, p=0.5), dict(temperature=0.01), dict(temperature=30.0)]:
        _check(x, g.random(4), **kw)


def test_masked_and_infinite_logits():
    low = np.finfo(np.float32).min
    rows = [[-INF] * 6, [NAN] * 6, [NAN, -INF, 2, NAN, 1, -INF], [low] * 6, [low, low, -INF, low, NAN, low],
            [1, INF, 2, INF, -INF, NAN], [INF] * 6, [low, 3e38, 0, -3e38, 3e38, 1], [-INF, -INF, -INF, -5, -INF, -INF],
            [0.0, -0.0, -1, -0.0, 0.0, -INF], [1e-45, 0, -1e-45, 1e-45, -INF, 1e-38]]
    for kw in SETTINGS:
        for u in (0.0, 0.45, 0.75, 1 - 2.0 ** -53):
            _check(np.array(rows, np.float32), u, **kw)


def test_temperatures_at_the_ends_of_their_range():
    g = rng(12)
    x = g.standard_normal((8, 5000)) * 4
    x[:, 7] = -INF
    x[4:, 9] = np.finfo(np.float32).min
    t = np.array([1e-45, 1e-30, 1e-6, 1e6, 1e30, 3.4e38, INF, 0.02], np.float32)
    for kw in [dict(), dict(k=30), dict(p=0.5), dict(min_p=0.5)]:
        _check(x, g.random(8), temperature=t, **kw)


def test_numbers_outside_their_range():
    x = rng(13).standard_normal((7, 300))
    for kw in [dict(), dict(k=10), dict(p=0.8)]:
        _check(x, [0.0, -1.0, NAN, 1.0, 7.0, INF, -INF], **kw)


def test_numbers_spread_evenly_draw_by_probability():
    """Over n numbers each token is drawn n p times, to within one."""
    import torch
    g = rng(14)
    n, V = 20000, 40
    row = (g.standard_normal(V) * 1.5).astype(np.float32)
    x = dev(np.broadcast_to(row, (n, V)).copy())
    u = dev((np.arange(n) + 0.5) / n)
    half = torch.full((n,), 0.7, device="cuda")
    z = np.exp(row.astype(np.float64) / np.float64(np.float32(0.7)))
    token, _ = S.sample(x, u, half)
    count = np.bincount(host(token), minlength=V)
    assert np.all(np.abs(count - n * z / z.sum()) <= 1)
    k = np.argsort(-z)[:6]
    token, _ = S.sample(x, u, half, torch.full((n,), 6, dtype=torch.int32, device="cuda"))
    count = np.bincount(host(token), minlength=V)
    assert np.all(np.abs(count[k] - n * z[k] / z[k].sum()) <= 1) and count.sum() == count[k].sum()


@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_rows_of_any_stride_and_alignment(xd):
    import torch
    g = rng(15)
    for W, first, V in [(1000, 0, 777), (1003, 1, 1000), (1001, 3, 990), (1008, 8, 1000), (4099, 2, 4097)]:
        t, x = _upload(g.standard_normal((5, W)) * 2, xd)
        cut, ref = t[:, first:first + V], x[:, first:first + V]
        _check(ref, g.random(5), k=20, t=cut)
        _check(ref, g.random(5), p=0.9, t=cut)
    one = t[2:3, 1:]                          # a row whose stride is never a step
    _check(x[2:3, 1:], [0.4], t=torch.as_strided(one, one.shape, (3, 1)))


def test_without_log_probabilities_and_with_buffers():
    import torch
    g = rng(16)
    t, x = _upload(g.standard_normal((6, 2500)), "f32")
    u = dev(g.random(6))
    a, none = S.sample(t, u)
    assert none is None
    st, n = S.bitlinear_sample_workspace_bytes(6, 2500)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((6,), -5, dtype=torch.int32, device="cuda")
    b, none = S.sample(t, u, out=(out, None), ws=ws)
    assert b is out and none is None and torch.equal(a, b)
    assert S.sample(t[:0], u[:0])[0].shape == (0,)


def test_the_same_in_every_run_and_on_another_stream():
    import torch
    g = rng(17)
    t, _ = _upload(g.standard_normal((20, 50000)), "f32")
    u, p = dev(g.random(20)), torch.full((20,), 0.95, device="cuda")
    first = S.sample(t, u, top_p=p, want_logprob=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            again = S.sample(t, u, top_p=p, want_logprob=True)
        both = S.sample(t, u, top_p=p, want_logprob=True)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, again)) and all(torch.equal(x, y) for x, y in zip(first, both))


def test_a_captured_draw():
    """Replays with other logits, numbers and settings between them."""
    import torch
    g = rng(18)
    B, V = 4, 9000
    x, u = torch.zeros(B, V, device="cuda"), torch.zeros(B, dtype=torch.float64, device="cuda")
    temp, k = torch.ones(B, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    token, lp = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda")
    ws = torch.empty(S.bitlinear_sample_workspace_bytes(B, V)[1], dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        S.sample(x, u, temp, k, out=(token, lp), ws=ws)
    for i in range(4):
        x.copy_(dev((g.standard_normal((B, V)) * 2).astype(np.float32)))
        if i == 2:
            x.fill_(0.5)
        u.copy_(dev(g.random(B)))
        temp.copy_(dev(g.choice([0, 0.5, 1.5], B).astype(np.float32)))
        k.copy_(dev(g.choice([0, 3, 6000], B).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        want = S.sample(x, u, temp, k, want_logprob=True)
        assert torch.equal(token, want[0]) and torch.equal(lp, want[1])
        for b in range(B):
            assert int(token[b]) == R.sample_row(host(x)[b], float(u[b]), float(temp[b]), int(k[b]))[0]


@pytest.mark.parametrize("V", [300, 40011, 131072])
@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("tail", ["equal", "narrow", "wide", "masked"])
def test_log_probabilities_of_confident_rows(V, xd, tail):
    """A token above a tail that weighs from a hundredth to ten times as much: the sum's error shows in a small result.
    A term of the sum is within 2^-33 of itself, so the sum's logarithm is off by 2^-33 tail / (1 + tail), at most 2^-33
    of the result; doubled for what fp64 adds, besides its roundings next to 1 (2^-50 for all of them); and the result is
    rounded once."""
    g = rng(V)
    x = {"equal": np.zeros((8, V)), "narrow": g.standard_normal((8, V)) * 0.05 - 0.37,
         "wide": g.standard_normal((8, V)) * 2 - 2, "masked": g.standard_normal((8, V)) * 0.3}[tail]
    if tail == "masked":
        x[:, ::3], x[:, 1::3] = -INF, np.finfo(np.float32).min
    x[:, V // 3] = np.log(V) + np.linspace(-2.3, 4.6, 8)
    t, x = _upload(x + 7.3, xd)
    import torch
    for temperature in (0.0, 0.7):
        token, lp = S.sample(t, dev(np.full(8, 0.3)), torch.full((8,), temperature, device="cuda"), want_logprob=True)
        token, lp = host(token), host(lp).astype(np.float64)
        for b in range(8):
            want, ref, _ = R.sample_row(x[b], 0.3, float(np.float32(temperature)))
            assert token[b] == want
            assert abs(lp[b] - ref) <= (2.0 ** -24 + 2.0 ** -32) * abs(ref) + 2.0 ** -50, (b, lp[b], ref)


@pytest.mark.parametrize("V,std,mask", [(262144, 0.5, None), (200000, 1.0, None), (131072, 1.0, -1e4),
                                        (131072, 1.0, np.finfo(np.float32).min), (131072, 1.0, -60.0)])
def test_wide_questions_of_large_rows(V, std, mask):
    """Top-k of a good part of the row and top-p behind it: together their bins hold more tokens than are listed, on
    flat rows, and where a finite mask or one far logit makes the bins wide."""
    g = rng(V + int(std * 10))
    x = g.standard_normal((2, V)) * std
    if mask == -60.0:
        x[:, 5] = mask
    elif mask is not None:
        x[g.random((2, V)) < 0.5] = mask
    for kw in [dict(k=V // 2, p=0.98), dict(k=V // 4, p=0.9), dict(p=0.95), dict(k=V // 2, p=0.95, min_p=0.05)]:
        _check(x, g.random(2), temperature=1.5, **kw)
