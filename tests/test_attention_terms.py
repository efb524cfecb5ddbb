"""That the bounds of the decode attention's accuracy tests tell three bf16 terms from two (CPU only): the
products are restated with either number of terms, on inputs whose leading two terms cancel."""
import numpy as np

import oracle.block_ref as R

U = 2.0 ** -24


def _cut(x, n):
    """fp32 values as n bf16 terms by truncation, summed in fp64."""
    rest, total = np.asarray(x, np.float32), np.zeros(np.shape(x))
    for _ in range(n):
        t = (rest.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        total += t
        rest = rest - t
    return total


def _leading(x):
    hi = R.bf16_round(x)
    return hi, R.bf16_round(x - hi)


def test_weights():
    """Weights 1, 1 and p on values -hi, -mid and 1, the bound that of six sums, an exponential and x's roundings."""
    x = np.random.default_rng(41).integers(1, 128, 64) / 128
    p = np.exp(-x).astype(np.float32)
    hi, mid = _leading(p)
    want = (np.exp(-x) - hi - mid) / (2 + np.exp(-x))
    bound = (3 * 0.37 + 2 + 6) / 2 * U + 2.0 ** -9 * np.abs(want)
    error = lambda n: np.abs((_cut(p, n) - hi.astype(np.float64) - mid) / (2 + p.astype(np.float64)) - want)
    assert np.all(error(3) <= bound) and np.mean(error(2) > bound) > 0.3


def test_queries():
    """A query (a, hi, mid) against keys 2^14 (1, -1, -1)."""
    a = (1 + np.random.default_rng(53).random((8, 16))).astype(np.float32)
    hi, mid = _leading(a)
    c = 2.0 ** 14
    want = c * (a.astype(np.float64) - hi - mid)
    bound = 3 * U * 2.0 ** 6 + 6 * U * np.abs(want)
    error = lambda n: np.abs(c * (_cut(a, n) - _cut(hi, n) - _cut(mid, n)) - want)
    assert np.all(error(3) <= bound) and np.mean(error(2) > bound) > 0.9


def test_three_terms_hold_24_bits():
    g = np.random.default_rng(3)
    x = (g.standard_normal(1000) * np.exp(g.uniform(-60, 60, 1000))).astype(np.float32)
    assert np.array_equal(_cut(x, 3), x.astype(np.float64))
    big = np.array([3.4028235e38, -3.4028235e38], np.float32)
    assert np.array_equal(_cut(big, 3), big.astype(np.float64)) and np.all(np.isinf(R.bf16_round(big)))
