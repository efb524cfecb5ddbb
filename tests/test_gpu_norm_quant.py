"""Residual + RMS norm + int8 quantization and its gradient against plain implementations.

The forward is defined to the bit (the mean square is summed in 64 bits, every other step is one
rounded fp32 operation), so int8 rows, scales, the stream and rstd must equal the reference's
exactly.  The gradient is held to a bound counted from its fp32 operations: u = 2^-24 per rounding,
a row's mean is a sum of at most 32 products per lane (three roundings each), 6 + 16 joining adds
and a division; a column's sum over T tokens rounds at most T + 24 times.
"""
import math

import numpy as np
import pytest

import oracle.block_ref as R
from parity_util import bf16_dev, dev, f32_bits, host
from synth import rng, to_bf16

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")
U = 2.0 ** -24


def _rows(g, T, K, dtype, scale=1.0):
    x = (g.standard_normal((T, K)) * scale).astype(np.float32)
    if dtype == "bf16":
        x, bits = to_bf16(x)
        return x, bf16_dev(bits)
    return x, dev(x)


def _f32(t):
    return host(t.float())


SIZES = [(1, 8), (1, 2560), (3, 512), (5, 520), (2, 4104), (1030, 264), (1025, 3200), (2, 8200),
         (1027, 1032), (1100, 2040), (1, 16384), (2, 32768), (7, 6912),
         (1029, 1000), (1026, 4104)]


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("xd,rd", [("f32", "bf16"), ("bf16", "f32"), ("bf16", "none"), ("f32", "f32"),
                                   ("bf16", "bf16"), ("f32", "none")])
def test_norm_quant_equals_definition(T, K, xd, rd):
    g = rng(T * 7 + K)
    x, xt = _rows(g, T, K, xd)
    res, rt = (None, None) if rd == "none" else _rows(g, T, K, rd, 3.0)
    w = (1 + 0.2 * g.standard_normal(K)).astype(np.float32)
    if T > 2:                       # a token of zeros, one with a single large value
        x[1] = 0
        xt[1] = 0
        if rt is not None:
            res[1] = 0
            rt[1] = 0
        x[2, K - 1] = -96.0
        xt[2, K - 1] = -96.0
    print(T, K, xd, rd, flush=True)
    q, sc, h, rstd = S.norm_quant(xt, dev(w), rt, eps=1e-5, want_rstd=True)
    q0, sc0, h0, r0 = R.norm_quant(x, w, res, 1e-5, 0, rd == "bf16")
    assert np.array_equal(f32_bits(_f32(h)), f32_bits(h0))
    assert np.array_equal(f32_bits(host(rstd)), f32_bits(r0))
    assert np.array_equal(host(q), q0)
    assert np.array_equal(f32_bits(host(sc)), f32_bits(sc0))
    if rd == "none":
        assert h is xt


@pytest.mark.parametrize("lift", [6, 8, 10, 12, 14, 16])
@pytest.mark.parametrize("T,mult", [(1, 5), (1029, 3), (3, 40)])
def test_norm_quant_lifted_rows(lift, T, mult):
    K = mult * lift * 8 // math.gcd(lift, 8)
    g = rng(lift + T)
    x, xt = _rows(g, T, K, "bf16")
    q, sc, _, rstd = S.norm_quant(xt, None, lift_M=lift)
    assert rstd is None
    q0, sc0, _, _ = R.norm_quant(x, None, None, 1e-6, lift)
    assert np.array_equal(host(q), q0) and np.array_equal(f32_bits(host(sc)), f32_bits(sc0))


def test_norm_quant_feeds_the_projection_like_act_quant():
    """The int8 rows are act_quant's of the normed rows, so a 2:4 projection reads them as they are."""
    g = rng(3)
    x, xt = _rows(g, 9, 1024, "f32")
    w = (1 + 0.1 * g.standard_normal(1024)).astype(np.float32)
    q, sc, _, rstd = S.norm_quant(xt, dev(w), want_rstd=True)
    n = (xt * rstd[:, None]) * dev(w)
    q1, sc1 = S.act_quant(n)
    assert np.array_equal(host(q), host(q1)) and np.array_equal(f32_bits(host(sc)), f32_bits(host(sc1)))


def test_norm_quant_in_place_on_another_stream_and_empty():
    import torch
    g = rng(4)
    x, xt = _rows(g, 33, 768, "f32")
    res, rt = _rows(g, 33, 768, "bf16")
    want = R.norm_quant(x, None, res, 1e-6, 0, True)
    q, sc = torch.empty(33, 768, dtype=torch.int8, device="cuda"), torch.empty(33, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        S.norm_quant(xt, None, rt, out=(q, sc, rt, None))       # the stream updated in place
    s.synchronize()
    assert np.array_equal(host(q), want[0])
    assert np.array_equal(f32_bits(_f32(rt)), f32_bits(want[2]))
    q, sc, h, r = S.norm_quant(xt[:0], None, rt[:0], want_rstd=True)
    assert q.shape == (0, 768) and sc.numel() == 0 and h.shape == (0, 768) and r.numel() == 0


def _grad_bound(dn, h, rstd, w, dres, out, grad):
    nh = np.abs(h * rstd[:, None].astype(np.float64))
    gw = np.abs(dn.astype(np.float64) * w)
    A = (gw * nh).mean(-1, keepdims=True)
    tol = rstd[:, None] * (4 * U * gw + nh * (62 * U) * A) + 4 * U * np.abs(out)
    if dres is not None:
        tol = tol + 2 * U * np.abs(dres)
    return tol + (2.0 ** -8 * np.abs(out) if grad == "bf16" else 0) + 1e-37


@pytest.mark.parametrize("T,K", [(1, 8), (3, 512), (17, 520), (130, 2048), (1031, 264), (5, 4096),
                                 (6, 4104), (3, 8192), (2, 16384), (2, 32768), (700, 3200),
                                 (2100, 2048), (20000, 256), (530, 8200), (300, 16384), (140, 32768),
                                 (900, 1000), (1500, 1928), (801, 5008)])
@pytest.mark.parametrize("dd,hd,gd,withres", [("f32", "bf16", "bf16", True), ("bf16", "f32", "f32", False),
                                              ("f32", "f32", "f32", True), ("bf16", "bf16", "bf16", False),
                                              ("f32", "bf16", "f32", True)])
def test_norm_grad_within_bound(T, K, dd, hd, gd, withres):
    g = rng(K + T)
    dn, dnt = _rows(g, T, K, dd, 2.0 ** -6)
    h, ht = _rows(g, T, K, hd, 2.0)
    dres, drt = _rows(g, T, K, gd, 2.0 ** -6) if withres else (None, None)
    w = (1 + 0.2 * g.standard_normal(K)).astype(np.float32)
    rstd = (1 / np.sqrt((h.astype(np.float64) ** 2).mean(-1) + 1e-6)).astype(np.float32)
    import torch
    print(T, K, dd, hd, gd, withres, flush=True)
    dh, dw = S.norm_quant_bwd(dnt, ht, dev(rstd), dev(w), drt,
                              dtype=torch.bfloat16 if gd == "bf16" else torch.float32)
    dh0, dw0 = R.norm_grad(dn, h, rstd, w, dres)
    assert np.all(np.abs(_f32(dh) - dh0) <= _grad_bound(dn, h, rstd, w, dres, dh0, gd))
    cols = (np.abs(dn.astype(np.float64)) * np.abs(h) * rstd[:, None]).sum(0)
    assert np.all(np.abs(host(dw) - dw0) <= (T + 26) * U * cols + 1e-37)
    again = S.norm_quant_bwd(dnt, ht, dev(rstd), dev(w), drt, dtype=dh.dtype)
    assert np.array_equal(f32_bits(host(again[1])), f32_bits(host(dw)))     # the order is fixed
    only, none = S.norm_quant_bwd(dnt, ht, dev(rstd), dev(w), drt, dtype=dh.dtype, want_dw=False)
    assert none is None and np.array_equal(f32_bits(_f32(only)), f32_bits(_f32(dh)))


def test_norm_grad_against_differences():
    """<dh, v> against a central difference of sum(dn * norm(h)) in 64 bits along v (and dw along a
    direction of the weight): the truncation error is far below the fp32 error allowed here."""
    g = rng(11)
    T, K, eps = 6, 640, 1e-3
    h, ht = _rows(g, T, K, "f32", 1.5)
    dn, dnt = _rows(g, T, K, "f32")
    w = (1 + 0.2 * g.standard_normal(K)).astype(np.float32)
    _, _, _, rstd = S.norm_quant(ht, dev(w), eps=eps, want_rstd=True)
    dh, dw = S.norm_quant_bwd(dnt, ht, rstd, dev(w))
    f = lambda hh, ww: float((dn.astype(np.float64) * R.norm_rows(hh, ww, eps)).sum())
    e = 1e-4
    for s in range(4):
        v = rng(50 + s).standard_normal((T, K))
        d = (f(h + e * v, w) - f(h - e * v, w)) / (2 * e)
        got = float((_f32(dh).astype(np.float64) * v).sum())
        assert abs(d - got) <= 1e-6 * np.abs(_f32(dh) * v).sum()
        u = rng(60 + s).standard_normal(K)
        d = (f(h, w + e * u) - f(h, w - e * u)) / (2 * e)
        assert abs(d - float((host(dw).astype(np.float64) * u).sum())) <= 1e-6 * np.abs(host(dw) * u).sum()


@pytest.mark.parametrize("T,K", [(20, 512), (300, 1032), (4200, 1032)])
def test_norm_grad_in_place_of_its_input(T, K):
    """dh over dn: dw still sums the gradient that came in."""
    g = rng(T)
    dn, dnt = _rows(g, T, K, "f32")
    h, ht = _rows(g, T, K, "bf16")
    rstd = dev((1 / np.sqrt((h.astype(np.float64) ** 2).mean(-1) + 1e-6)).astype(np.float32))
    want, dw = S.norm_quant_bwd(dnt, ht, rstd)
    keep = f32_bits(host(want)).copy()
    got, dw1 = S.norm_quant_bwd(dnt, ht, rstd, out=(dnt, dw.clone()))
    assert got is dnt and np.array_equal(f32_bits(host(dnt)), keep)
    assert np.array_equal(f32_bits(host(dw)), f32_bits(host(dw1)))


def test_norm_grad_in_place_and_no_tokens():
    g = rng(12)
    dn, dnt = _rows(g, 20, 512, "f32")
    h, ht = _rows(g, 20, 512, "bf16")
    rstd = dev((1 / np.sqrt((h ** 2).mean(-1) + 1e-6)).astype(np.float32))
    dres, drt = _rows(g, 20, 512, "f32")
    want, dw0 = S.norm_quant_bwd(dnt, ht, rstd, None, drt)
    keep = want.clone()
    got, dw1 = S.norm_quant_bwd(dnt, ht, rstd, None, drt, out=(drt, dw0.clone()))
    assert got is drt and np.array_equal(f32_bits(host(drt)), f32_bits(host(keep)))
    assert np.array_equal(f32_bits(host(dw0)), f32_bits(host(dw1)))
    dh, dw = S.norm_quant_bwd(dnt[:0], ht[:0], rstd[:0])
    assert dh.shape == (0, 512) and not host(dw).any()
