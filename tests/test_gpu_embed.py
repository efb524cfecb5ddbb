"""Embedding rows to the bit, and their gradient against sums in fp64.

The gradient's bound: a row that n tokens name is a sum of n fp32 terms in some order of additions (at
most n - 1 roundings on a term's way, plus one product by the scale and, accumulating, one addition):
|error| <= (n + 1) u * sum |terms| with u = 2^-24, to first order; (1 + 2^-8) covers the second.
"""
import numpy as np
import pytest

import oracle.block_ref as BR
import oracle.step_ref as R
from parity_util import dev, f32_bits, host
from synth import rng

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")

U = 2.0 ** -24


def _float(g, shape, dtype, std=1.0):
    """(device tensor, its fp32 values)."""
    x = (g.standard_normal(shape) * std).astype(np.float32)
    t = dev(x)
    if dtype == "bf16":
        t = t.bfloat16()
        x = BR.bf16_round(x)
    return t, x


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


@pytest.mark.parametrize("T,V,K", [(1, 1, 8), (1, 100, 2560), (5, 33, 64), (16, 1000, 3200), (37, 50, 2048),
                                   (4, 7, 2056), (3, 5, 16384), (2, 3, 32768), (1021, 777, 104)])
@pytest.mark.parametrize("td,yd", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("scale", [1.0, 0.3, 50.5966])
def test_rows(T, V, K, td, yd, scale):
    g = rng(T + V + K)
    table, ref = _float(g, (V, K), td)
    ids = g.integers(0, V, T).astype(np.int32)
    if T > 4:
        ids[1], ids[2], ids[3] = -1, -2 ** 31, V - 1
        ids[4] = V + 5 if T > 16 else V - 1
    y = S.embed(dev(ids), table, scale=scale, dtype=_dt(yd))
    want = R.embed(ids, ref, scale)
    got = host(y.float())
    if yd == "bf16":
        ok = ~np.isnan(want)
        want = np.where(ok, BR.bf16_round(np.where(ok, want, 0)), np.nan)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(f32_bits(got[~nan]), f32_bits(want[~nan].astype(np.float32)))


def test_rows_of_a_table_past_4_gib():
    """Offsets that pass 32 bits, in bytes and in elements."""
    import torch
    V, K = 140000, 32768                     # 4.6e9 elements, bf16
    table = torch.empty(V, K, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, 70000, 131071, 131072, V - 1, 65536], dtype=torch.int32, device="cuda")
    table[ids.long()] = torch.randn(6, K, device="cuda").bfloat16()
    y = S.embed(ids, table)
    assert torch.equal(y, table[ids.long()])


def test_no_tokens():
    import torch
    t = torch.zeros(4, 64, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert S.embed(none, t).shape == (0, 64)
    assert not S.embed_bwd(torch.zeros(0, 64, device="cuda"), none, 9).any()
    kept = torch.ones(9, 64, device="cuda")
    S.embed_bwd(torch.zeros(0, 64, device="cuda"), none, 9, accumulate=True, out=kept)
    assert bool((kept == 1).all())


def _ids(g, T, V, kind):
    if kind == "one":
        return np.full(T, V // 2, np.int32)
    if kind == "even":
        return g.integers(0, V, T).astype(np.int32)
    if kind == "runs":                       # lengths around what a wave takes and what it sums alone
        n = [1, 2, 15, 16, 17, 31, 32, 33, 34, 47, 48, 49, 63, 64, 65, 130]
        ids = np.repeat(np.arange(len(n)), n)[:T] % V
        ids = np.concatenate((ids, g.integers(0, V, T - len(ids)))).astype(np.int32)
        return g.permutation(ids).astype(np.int32)
    ids = np.minimum((V + 1.0) ** g.random(T) - 1, V - 1).astype(np.int32)
    if kind == "padded":
        ids[g.random(T) < 0.4] = -1
        ids[g.random(T) < 0.05] = V
    return ids


def _grad_check(g, T, V, K, dd, kind, scale=1.0, accum=False):
    dy, ref = _float(g, (T, K), dd, 2.0 ** -6)
    ids = _ids(g, T, V, kind)
    into = (g.standard_normal((V, K)) * 2.0 ** -6).astype(np.float32) if accum else None
    print(T, V, K, dd, kind, accum, flush=True)
    out = dev(into) if accum else None
    if not accum:
        import torch
        out = torch.full((V, K), float("nan"), device="cuda")
    got = host(S.embed_bwd(dy, dev(ids), V, scale=scale, accumulate=accum, out=out)).astype(np.float64)
    want, mag, n = R.embed_grad(ref, ids, V, float(np.float32(scale)), into)
    err = np.abs(got - want)
    assert np.all(err <= (n[:, None] + 1) * U * mag * (1 + 2.0 ** -8)), (err / (mag + 1e-30)).max()
    none = n == 0
    assert np.array_equal(got[none], into[none].astype(np.float64) if accum else np.zeros_like(got[none]))
    return got


@pytest.mark.parametrize("T,V,K", [(1, 1, 8), (2, 5, 64), (16, 9, 512), (17, 300, 520), (33, 2, 256), (100, 40, 1032),
                                   (1000, 5000, 136), (1024, 70, 64), (1025, 70, 64), (3000, 900, 264)])
@pytest.mark.parametrize("dd", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["one", "even", "zipf", "padded"])
@pytest.mark.parametrize("accum", [False, True])
def test_gradient(T, V, K, dd, kind, accum):
    _grad_check(rng(T + V + K), T, V, K, dd, kind, 1.0 if K % 16 else 7.25, accum)


@pytest.mark.parametrize("T", [700, 900, 2100, 5003])
@pytest.mark.parametrize("dd", ["f32", "bf16"])
@pytest.mark.parametrize("accum", [False, True])
def test_gradient_of_runs_of_every_kind(T, dd, accum):
    for seed in range(3):
        _grad_check(rng(seed + T), T, 40, 72, dd, "runs", 1.0, accum)


@pytest.mark.parametrize("T,V,K,kind", [(16384, 31, 64, "zipf"), (16385, 5000, 64, "padded"), (40000, 3, 8, "even"),
                                        (100003, 20000, 16, "zipf"), (65536, 900, 8, "padded"), (65537, 70, 8, "zipf"),
                                        (131073, 5, 8, "padded"), (200001, 100000, 8, "even"),
                                        (400000, 1 << 21, 8, "padded")])
def test_gradient_of_many_tokens(T, V, K, kind):
    """One span of chunks and several, and rows of ten thousand tokens."""
    _grad_check(rng(T), T, V, K, "bf16", kind)


@pytest.mark.parametrize("V", [(1 << 21) - 1, 1 << 21, (1 << 24) + 3])
@pytest.mark.parametrize("accum", [False, True])
def test_gradient_of_tables_of_many_rows(V, accum):
    """Around the change of the sort's keys, first and last rows among the tokens'."""
    import torch
    g = rng(V)
    T, K = 3000, 8
    ids = g.integers(0, V, T).astype(np.int32)
    ids[:40] = [0, V - 1, V - 2, 1] * 10
    ids[50:90] = -1
    ids[90:130] = np.minimum(V + np.arange(40), 2 ** 31 - 1)
    dy, ref = _float(g, (T, K), "f32")
    out = torch.ones((V, K), device="cuda") if accum else torch.full((V, K), float("nan"), device="cuda")
    out = S.embed_bwd(dy, dev(ids), V, accumulate=accum, out=out)
    ok = (ids >= 0) & (ids < V)
    rows, at = np.unique(ids[ok], return_inverse=True)
    want, mag = np.full((len(rows), K), float(accum)), np.full((len(rows), K), float(accum))
    np.add.at(want, at, ref[ok].astype(np.float64))
    np.add.at(mag, at, np.abs(ref[ok].astype(np.float64)))
    index = torch.from_numpy(rows).cuda().long()
    got = host(out[index]).astype(np.float64)
    n = np.bincount(at)[:, None]
    assert np.all(np.abs(got - want) <= (n + 1) * U * mag * (1 + 2.0 ** -8))
    out[index] = float(accum)
    assert bool((out == float(accum)).all())


def test_gradient_where_no_id_has_a_row():
    import torch
    ids = torch.tensor([-1, 9, 2 ** 31 - 1, -7] * 20, dtype=torch.int32, device="cuda")
    out = torch.full((9, 64), float("nan"), device="cuda")
    assert not S.embed_bwd(torch.full((80, 64), float("nan"), device="cuda"), ids, 9, out=out).any()


def test_gradient_keeps_infinite_and_nan_rows_to_themselves():
    import torch
    dy = torch.ones(100, 64, device="cuda")
    ids = (torch.arange(100, device="cuda") % 5).int()
    dy[ids == 2] = float("inf")
    dy[3] = float("nan")
    got = S.embed_bwd(dy, ids, 6)
    assert bool((got[[0, 1, 4]] == 20).all()) and bool(torch.isinf(got[2]).all()) and bool(torch.isnan(got[3]).all())
    assert not got[5].any()


def test_gradient_does_not_vary_from_run_to_run():
    import torch
    g = rng(3)
    dy, _ = _float(g, (5000, 256), "f32")
    ids = dev(_ids(g, 5000, 300, "zipf"))
    ws = torch.randint(0, 255, (S.bitlinear_embed_bwd_workspace_bytes(5000, 256)[1],), dtype=torch.uint8, device="cuda")
    first = S.embed_bwd(dy, ids, 300, ws=ws)
    for _ in range(5):
        assert torch.equal(first, S.embed_bwd(dy, ids, 300, ws=ws))


def test_gradient_against_differences():
    """Of sum(embed(table) * c): the table's gradient is that of the formula, direction by direction."""
    import torch
    g = rng(8)
    T, V, K, scale = 60, 11, 64, 3.5
    table, t = _float(g, (V, K), "f32")
    c, cr = _float(g, (T, K), "f32")
    ids = _ids(g, T, V, "padded")
    d = host(S.embed_bwd(c, dev(ids), V, scale=scale)).astype(np.float64)
    for _ in range(8):
        v = g.standard_normal((V, K)).astype(np.float32) * 0.5
        f = [(host(S.embed(dev(np.where(ids >= V, -1, ids)), dev(t + s * v), scale=scale)).astype(np.float64) * cr).sum()
             for s in (1.0, -1.0)]
        # linear in the table: the central difference is exact but for the roundings of t +- v and of y
        bound = 4 * U * scale * np.abs(cr).sum() * (np.abs(t).max() + np.abs(v).max())
        assert abs((f[0] - f[1]) / 2 - (d * v).sum()) <= bound + 1e-5 * (np.abs(d) * np.abs(v)).sum()


@pytest.mark.parametrize("accum", [False, True])
def test_a_captured_gradient(accum):
    """Replays with other gradients and ids between them; a run of many tokens in some."""
    import torch
    g = rng(21)
    T, V, K = 1500, 60, 128
    dy, ids = torch.empty(T, K, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    out = torch.zeros(V, K, device="cuda")
    ws = torch.empty(S.bitlinear_embed_bwd_workspace_bytes(T, K)[1], dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        S.embed_bwd(dy, ids, V, accumulate=accum, out=out, ws=ws)
    for kind in ("zipf", "one", "even", "padded"):
        dy.copy_(_float(g, (T, K), "f32")[0])
        ids.copy_(dev(_ids(g, T, V, kind)))
        eager = S.embed_bwd(dy, ids, V, accumulate=accum, out=out.clone())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("T,V,K,kind", [(1, 70000, 1024, "even"), (33, 70000, 1024, "one"), (2047, 30000, 2056, "zipf"),
                                        (3749, 30000, 2056, "padded"), (3750, 30000, 2056, "even"), (3751, 30000, 2056, "even"),
                                        (8750, 70000, 1024, "runs"), (70000, 560000, 104, "padded"), (5, 8, 32768, "even"),
                                        (4100, (1 << 21) + 5, 40, "zipf"), (9, 2000, 32768, "even")])
def test_gradient_of_large_tables(T, V, K, kind):
    """Few tokens over tables of hundreds of MB, on both sides of what clears them first: rows at their places, the last
    and the first row among them, everything else zero."""
    import torch
    g = rng(T + V)
    ids = _ids(g, T, V, kind)
    ids[-1], ids[T // 2] = V - 1, 0
    dy, ref = _float(g, (T, K), "bf16", 2.0 ** -6)
    print(T, V, K, kind, flush=True)
    out = S.embed_bwd(dy, dev(ids), V, scale=3.0, out=torch.full((V, K), float("nan"), device="cuda"))
    ok = (ids >= 0) & (ids < V)
    rows, at = np.unique(ids[ok], return_inverse=True)
    want, mag, n = R.embed_grad(ref[ok], at, len(rows), 3.0)
    index = torch.from_numpy(rows).cuda().long()
    got = host(out[index]).astype(np.float64)
    assert np.all(np.abs(got - want) <= (n[:, None] + 1) * U * mag * (1 + 2.0 ** -8))
    out[index] = 0
    assert bool((out == 0).all())
