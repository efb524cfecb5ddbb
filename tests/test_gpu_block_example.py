"""The example's decode steps and training step, stage by stage against the plain implementations: each
stage is checked on the inputs it had, so every output keeps its own bar (int8 rows, scales and rotated
queries to the bit, projections within the fp32 rescale, attention within its counted bound)."""
import os
import sys

import numpy as np
import pytest

import oracle as O
import oracle.block_ref as R
from parity_util import assert_y_close, f32_bits, host

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _f(t):
    return host(t.float())


def _same(a, b):
    return np.array_equal(f32_bits(a), f32_bits(b))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_decode_steps(kv):
    import torch

    import block as E
    seqs, hidden, heads, kvh, D, ffn, page = 5, 256, 4, 2, 64, 320, 4
    b = E.DecodeBlock(seqs, hidden, heads, kvh, D, ffn, page, max_len=20, kv=kv, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    b.stream.copy_(torch.randn(seqs, hidden, generator=g, device="cuda"))
    delta = torch.randn(seqs, hidden, generator=g, device="cuda")
    start = torch.tensor([0, 3, -2, 0, 7], dtype=torch.int32, device="cuda")   # the third begins as padding
    table = host(b.table)
    for t in range(9):
        pos = start + t
        lens = (pos + 1).clamp(min=0).int()
        trace = []
        kc0, vc0 = b.k_cache.clone(), b.v_cache.clone()
        delta = b.step(delta, pos, lens, trace)
        tr = dict(trace)
        x, stream = (_f(v) for v in tr["in"])
        xq, sc, h, q, k, v = tr["qkv"]
        q0, s0, h0, _ = R.norm_quant(x, host(b.w1), stream, 1e-6, 0, True)
        assert np.array_equal(host(xq), q0) and _same(host(sc), s0) and _same(_f(h), h0)
        # rotated queries and the appended rows
        qr = R.bf16_round(R.rope(_f(q).reshape(seqs, heads, D), host(pos), table))
        assert _same(_f(tr["attn"][0]), qr)
        kr = R.rope(_f(k).reshape(seqs, kvh, D), host(pos), table)
        vr = _f(v).reshape(seqs, kvh, D)
        kc, vc, blocks = _f(kc0), _f(vc0), host(b.blocks)
        for s in range(seqs):
            p = int(pos[s])
            if p < 0:
                continue
            pg, off = blocks[s, p // page], p % page
            if kv == "bf16":
                kc[pg, :, off], vc[pg, :, off] = R.bf16_round(kr[s]), R.bf16_round(vr[s])
            else:
                (kc[pg, :, off], ks), (vc[pg, :, off], vs) = O.act_quant(kr[s]), O.act_quant(vr[s])
                assert _same(host(b.scales["k_scale"])[pg, :, off], ks)
                assert _same(host(b.scales["v_scale"])[pg, :, off], vs)
        assert _same(_f(b.k_cache), kc) and _same(_f(b.v_cache), vc)
        scales = {} if kv == "bf16" else dict(ks=host(b.scales["k_scale"]), vs=host(b.scales["v_scale"]))
        want, _, mag, smag = R.paged_attn(qr, kc, vc, blocks, host(lens), D ** -0.5, **scales)
        u = 2.0 ** -24
        e = ((D + 6) * u * smag + 4 * u + 2.0 ** -17 + 84 * u)[..., None]
        got = _f(tr["attn"][1])
        assert np.all(np.abs(got - want) <= 2 * e * mag + 2.0 ** -8 * np.abs(want) + 1e-30)
        # the output projection's input is act_quant's of the attention's output
        oq, os_ = O.act_quant(got.reshape(seqs, -1))
        assert np.array_equal(host(tr["o"][0]), oq) and _same(host(tr["o"][1]), os_)
        xq, sc, h, gate, up = tr["gate_up"]
        q0, s0, h0, _ = R.norm_quant(_f(tr["o"][2]), host(b.w2), h0, 1e-6, 0, True)
        assert np.array_equal(host(xq), q0) and _same(host(sc), s0) and _same(_f(h), h0)
        inner, xq, sc, y = tr["down"]
        q0, s0, _, _ = R.norm_quant(_f(inner), host(b.w3))
        assert np.array_equal(host(xq), q0) and _same(host(sc), s0)
        assert np.isfinite(_f(y)).all() and _same(_f(delta), _f(y))


def test_decode_step_as_a_graph():
    """Replays of a captured step, positions and lengths advanced between them, equal eager steps."""
    import torch

    import block as E
    runs = []
    for graphed in (False, True):
        b = E.DecodeBlock(4, 256, 4, 2, 64, 320, 4, max_len=200, kv="bf16", seed=7)
        g = torch.Generator(device="cuda")
        g.manual_seed(6)
        b.stream.copy_(torch.randn(4, 256, generator=g, device="cuda"))
        delta = torch.randn(4, 256, generator=g, device="cuda")
        pos = torch.tensor([0, 150, 30, 140], dtype=torch.int32, device="cuda")
        lens = pos + 1
        torch.cuda.synchronize()
        out = []
        if graphed:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=torch.cuda.Stream()):
                delta.copy_(b.step(delta, pos, lens))
        for _ in range(6):
            if graphed:
                gr.replay()
            else:
                delta = b.step(delta, pos, lens).clone()
            torch.cuda.synchronize()
            out.append(host(delta).copy())
            pos += 1
            lens += 1
        runs.append(out)
    for x, y in zip(*runs):
        assert np.isfinite(x).all() and _same(x, y)


def test_training_step():
    import block as E
    T, hidden, heads, D = 48, 256, 2, 128
    r = E.train_attention_input(T, hidden, heads, D, seed=9)
    ref = O.pack(host(r["W"]), 2, 4)
    q0, s0, h0, r0 = R.norm_quant(_f(r["x"]), host(r["w"]), _f(r["res"]), 1e-6, 0, True)
    assert np.array_equal(host(r["xq"]), q0) and _same(host(r["scale"]), s0) and _same(host(r["rstd"]), r0)
    assert_y_close(host(r["y"]), O.rescale(O.acc_dense(ref["W_eff"], q0), ref["gamma"], s0))
    pos, table = host(r["pos"]), host(r["table"])
    assert _same(_f(r["q"]), R.bf16_round(R.rope(host(r["y"]).reshape(T, heads, D), pos, table)))
    assert _same(_f(r["dy"]), R.bf16_round(R.rope(_f(r["dq"]), pos, table, inverse=True)))
    dn0, dW0 = O.backward(_f(r["dy"]).reshape(T, -1), ref["W_eff"], ref["gamma"], q0, s0)
    # fp32 sums over the reduction axis: at most (terms + 4) roundings of the sum of magnitudes
    u = 2.0 ** -24
    n = heads * D
    mag, _ = O.backward(np.abs(_f(r["dy"])).reshape(T, -1), np.abs(ref["W_eff"]), ref["gamma"], q0, s0)
    assert np.all(np.abs(host(r["dn"]) - dn0) <= (n + 4) * u * np.abs(mag) + 1e-30)
    dh0, dw0 = R.norm_grad(host(r["dn"]), h0, r0, host(r["w"]), _f(r["dstream"]))
    assert np.linalg.norm(_f(r["dh"]) - dh0) <= 2.0 ** -8 * np.linalg.norm(dh0)
    assert np.linalg.norm(host(r["dw"]) - dw0) <= T * u * np.linalg.norm(
        (np.abs(host(r["dn"])) * np.abs(h0) * r0[:, None]).sum(0))
