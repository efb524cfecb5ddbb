"""4-bit weights: codes and scales to the bit, products against sums in fp64.

A group's inner sum is exact.  Joining n groups takes at most n fused multiply-adds on a term's way, up to 7
additions where waves share the columns, and the product by the token's scale: |error| <= (n + 8) u * sum over
groups |s acc| * x_scale to first order, u = 2^-24; (1 + 2^-8) covers the second.
"""
import numpy as np
import pytest

import oracle.block_ref as BR
import oracle.step_ref as R
from parity_util import dev, host
from synth import rng

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")

U = 2.0 ** -24


def _weights(g, n, K, kind="normal"):
    W = (g.standard_normal((n, K)) * 0.02).astype(np.float32)
    if kind == "spread":                     # every magnitude from denormal to the largest
        W *= np.exp2(g.integers(-140, 128, (n, K // 32))).astype(np.float32).repeat(32, 1)
        W = np.clip(W, -3.3e38, 3.3e38)
    if kind == "ties":                       # quotients on and beside halves
        W = (g.integers(-14, 15, (n, K)) * 0.5).astype(np.float32)
        W[:, ::32] = 7.0
    if kind == "zeros":
        W[g.random((n, K // 32)).repeat(32, 1) < 0.5] = 0.0
        W[0] = -0.0
    return W


def _bits(t):
    import torch
    return host(t.view(torch.int16)).view(np.uint16)


@pytest.mark.parametrize("n,K", [(1, 128), (16, 128), (17, 256), (5, 384), (100, 640), (33, 2560), (3, 8192)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("wd", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "spread", "ties", "zeros"])
def test_packing(n, K, group, wd, kind):
    W = _weights(rng(n + K + group), n, K, kind)
    t = dev(W)
    if wd == "bf16":
        t, W = t.bfloat16(), BR.bf16_round(W)
    codes, scales = S.q4_pack(t, group)
    c, s = R.q4_pack(*R.q4_quantize(W, group), group)
    assert np.array_equal(_bits(scales), s)
    assert np.array_equal(host(codes), c)


@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (160, 32), (64, 64), (192, 64), (4160, 64)])
def test_packing_of_columns_that_end_inside_a_block(K, group):
    import torch
    W = _weights(rng(K), 20, K)
    st, cb, sb = S.bitlinear_q4_bytes(20, K, group)
    out = (torch.full((cb,), 255, dtype=torch.uint8, device="cuda"),
           torch.full((sb // 2,), float("nan"), dtype=torch.bfloat16, device="cuda"))
    codes, scales = S.q4_pack(dev(W), group, out=out)
    c, s = R.q4_pack(*R.q4_quantize(W, group), group)
    assert np.array_equal(host(codes), c) and np.array_equal(_bits(scales), s)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_groups_that_are_not_finite(bad):
    """Their scale is NaN, and the products of their rows, and of no others."""
    W = _weights(rng(4), 40, 256)
    W[7, 130], W[33, 5] = bad, bad
    codes, scales = S.q4_pack(dev(W), 64)
    c, s = R.q4_pack(*R.q4_quantize(W, 64), 64)
    assert np.array_equal(host(codes), c) and np.array_equal(_bits(scales), s)
    xq, xs = dev(np.zeros((3, 256), np.int8)), dev(np.ones(3, np.float32))
    y = host(S.q4_fwd(xq, xs, 256, codes, scales, 40))
    nan = np.isnan(y)
    assert nan[:, [7, 33]].all() and nan.sum() == 6 and not y[~nan].any()


def _case(g, T, n, K, group, xmax=127):
    W = _weights(g, n, K)
    q, s = R.q4_quantize(W, group)
    codes, scales = S.q4_pack(dev(W), group)
    xq = np.clip(np.rint(g.standard_normal((T, K)) * 40), -xmax, xmax).astype(np.int8)
    xs = (0.01 + g.random(T)).astype(np.float32)
    return xq, xs, q, s, codes, scales


def _check(y, xq, xs, q, s, group):
    want, mag = R.q4_forward(xq, xs, q, s, group)
    err = np.abs(y.astype(np.float64) - want)
    bound = (q.shape[1] // group + 8) * U * mag * (1 + 2.0 ** -8)
    assert np.all(err <= bound), (err / (bound + 1e-300)).max()


@pytest.mark.parametrize("T", [1, 2, 4, 5, 15, 16, 17, 31, 33, 48, 49, 64, 65, 130, 200])
@pytest.mark.parametrize("n,K,group", [(1, 32, 32), (15, 96, 32), (48, 128, 128), (100, 640, 64), (257, 1280, 32),
                                       (1000, 2560, 64), (513, 6912, 128), (130, 192, 64)])
def test_products(T, n, K, group):
    import torch
    xq, xs, q, s, codes, scales = _case(rng(T + n + K), T, n, K, group)
    print(T, n, K, group, flush=True)
    out = torch.full((T, n), float("nan"), device="cuda")
    _check(host(S.q4_fwd(dev(xq), dev(xs), K, codes, scales, n, group, out=out)), xq, xs, q, s, group)


@pytest.mark.parametrize("T,n,K,group", [(1, 40000, 256, 64), (3, 33333, 512, 128), (40, 70001, 128, 32), (64, 8200, 4224, 64),
                                         (9, 50, 65536, 128), (64, 50, 16384, 32), (1, 17000, 4096, 32),
                                         (16, 8208, 1024, 64), (5, 33000, 256, 64), (30, 20000, 640, 32),
                                         (48, 17000, 512, 128), (48, 9000, 1152, 32), (20, 33000, 384, 128)])
def test_products_of_many_rows_or_columns(T, n, K, group):
    """One, two, four and eight waves per tile, several parts of K in LDS, spare tiles at the end."""
    xq, xs, q, s, codes, scales = _case(rng(n + K), T, n, K, group)
    _check(host(S.q4_fwd(dev(xq), dev(xs), K, codes, scales, n, group)), xq, xs, q, s, group)


def test_products_at_the_ends_of_int8():
    """Every product at its largest, -128 among the rows: the inner sums stay exact."""
    for group in (32, 64, 128):
        q = np.where(np.arange(256) % 2 == 0, -7, 7).astype(np.int8)[None].repeat(20, 0)
        codes, scales = S.q4_pack(dev(q.astype(np.float32)), group)
        xq = np.where(q[:2] < 0, -128, 127).astype(np.int8)
        y = host(S.q4_fwd(dev(xq), dev(np.ones(2, np.float32)), 256, codes, scales, 20, group))
        assert np.all(y == 128 * 7 * (128 + 127))


def test_tokens_do_not_touch_each_other():
    """A token's products are its own to the bit, whatever rows stand beside it."""
    import torch
    xq, xs, q, s, codes, scales = _case(rng(77), 16, 300, 512, 64)
    y = S.q4_fwd(dev(xq), dev(xs), 512, codes, scales, 300)
    for t in range(16):
        assert torch.equal(y[t:t + 1], S.q4_fwd(dev(xq[t:t + 1]), dev(xs[t:t + 1]), 512, codes, scales, 300))


def test_no_tokens():
    import torch
    codes, scales = S.q4_pack(torch.zeros(8, 64, device="cuda"), 64)
    y = S.q4_fwd(torch.zeros(0, 64, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda"), 64, codes, scales, 8)
    assert y.shape == (0, 8)


def test_a_captured_product():
    import torch
    g = rng(5)
    xq, xs, q, s, codes, scales = _case(g, 5, 200, 640, 32)
    x, sc, y = dev(xq), dev(xs), torch.zeros(5, 200, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        S.q4_fwd(x, sc, 640, codes, scales, 200, 32, out=y)
    for _ in range(3):
        xq = np.clip(np.rint(g.standard_normal((5, 640)) * 40), -127, 127).astype(np.int8)
        x.copy_(dev(xq))
        graph.replay()
        _check(host(y), xq, xs, q, s, 32)


@pytest.mark.parametrize("T", [1, 4, 5, 20, 40, 64])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_products_of_the_largest_weights_and_the_smallest_scales(T, group):
    """Sums of groups up to fp32's largest number, and scales of tokens below its normal ones: as long as the joined sum
    is finite and the result normal, the bound is that of any other product."""
    g = rng(T + group)
    n, K = 40, 512
    W = _weights(g, n, K)
    top = np.float32(3.2e38) * np.exp2(-g.integers(0, 6, n)).astype(np.float32)
    W[:, :group] = 0.0
    W[np.arange(n), g.integers(0, group, n)] = top * g.choice([-1, 1], n)     # code 7 or -7, scale of top / 7
    q, s = R.q4_quantize(W, group)
    codes, scales = S.q4_pack(dev(W), group)
    xq = g.integers(-127, 128, (T, K)).astype(np.int8)
    xq[:, :group] = g.choice([-1, 1], (T, 1))
    assert np.abs(s[:, 0] * 7).max() < np.finfo(np.float32).max * (1 - 2.0 ** -8)
    for xs in (0.01 + g.random(T), (1 + g.random(T)) * 2.0 ** -126, np.ldexp(1 + g.integers(0, 32, T) / 32, -140)):
        xs = xs.astype(np.float32)
        _check(host(S.q4_fwd(dev(xq), dev(xs), K, codes, scales, n, group)), xq, xs, q, s, group)


@pytest.mark.parametrize("T", [1, 2, 4, 5, 16, 32, 48, 64, 65])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("code,x", [(-8, -128), (-8, 127), (7, 127), (7, -128), (-7, -128)])
def test_inner_sums_at_their_ends(T, group, code, x):
    """The largest groups' sums, codes of -8 written into the layout among them: whole numbers below 2^24, so exact."""
    n, K = 40, 512
    q = np.full((n, K), code, np.int8)
    q[::3, ::2] = 0
    codes, scales = R.q4_pack(q, np.ones((n, K // group), np.float32), group)
    xq = np.full((T, K), x, np.int8)
    xq[1::2, 1::2] = -x - 1                                # -128 and 127 in turn
    import torch
    y = host(S.q4_fwd(dev(xq), dev(np.ones(T, np.float32)), K, dev(codes),
                      dev(scales.view(np.int16)).view(torch.bfloat16), n, group))
    assert np.array_equal(y, xq.astype(np.int64) @ q.T.astype(np.int64))


@pytest.mark.parametrize("T", [3, 16, 30, 48, 64, 100])
@pytest.mark.parametrize("n,K", [(300, 512), (2560, 1280), (9000, 256)])
def test_other_tokens_of_a_call_do_not_touch_a_token(T, n, K):
    """At one number of tokens, whatever the other rows and scales of the call are: NaN scales and full rows too."""
    import torch
    g = rng(T + n)
    xq, xs, q, s, codes, scales = _case(g, T, n, K, 64)
    first = S.q4_fwd(dev(xq), dev(xs), K, codes, scales, n)
    _check(host(first), xq, xs, q, s, 64)
    for t in sorted({0, 1, T // 2, T - 1}):
        other, os = g.integers(-128, 128, (T, K)).astype(np.int8), np.full(T, np.nan, np.float32)
        other[t], os[t] = xq[t], xs[t]
        assert torch.equal(first[t], S.q4_fwd(dev(other), dev(os), K, codes, scales, n)[t])
