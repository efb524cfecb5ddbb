"""The example's steps from token ids to token ids, stage by stage against the plain implementations on the inputs
that each stage had: tables, embedding rows, int8 rows and tokens to the bit, logits within the joined groups'
bound; the gradients of its training half against the formulas and against differences.  And the tables in front
of the cache's own calls: prompts appended by kv_step's rows, and attended."""
import os
import sys

import numpy as np
import pytest

import oracle as O
import oracle.block_ref as BR
import oracle.step_ref as R
from parity_util import dev, f32_bits, host
from synth import rng

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

U = 2.0 ** -24


def _same(a, b):
    return np.array_equal(f32_bits(a), f32_bits(b))


def _model(seed, **kw):
    import torch

    import model as E
    m = E.Model(6, layers=2, vocab=1003, hidden=256, heads=4, kv_heads=2, D=64, ffn=320, page=4, max_len=24, seed=seed,
                **kw)
    g = rng(seed)
    m.tokens.copy_(dev(g.integers(0, 1003, 6).astype(np.int32)))
    m.settings["temperature"].copy_(torch.tensor([0.0, 0.5, 0.8, 1.0, 1.5, 0.7]))
    m.settings["top_k"].copy_(torch.tensor([0, 0, 5, 50, 300, 2]))
    m.settings["top_p"].copy_(torch.tensor([1.0, 0.9, 1.0, 0.95, 0.5, 1.0]))
    return m, g


FRESH = [[1] * 6, [1] * 6, [1, 1, -1, 1, 0, 1], [1] * 6, [-1, 1, 1, 1, 1, -1], [1] * 6, [0, 1, 1, 0, 1, 1], [1] * 6]


@pytest.mark.parametrize("group,pages", [(64, None), (128, 9), (32, 14)])
def test_steps(group, pages):
    """pages: too few for all requests, which then wait."""
    m, g = _model(3, group=group, pages=pages)
    W = None
    for t in range(16):
        m.fresh.copy_(dev(np.array(FRESH[t % len(FRESH)], np.int32)))
        u = g.random(6)
        m.u.copy_(dev(u))
        trace = []
        m.step(trace)
        tr = {n: [host(x.float() if x.dtype.is_floating_point else x) for x in v] for n, v in trace}
        lens, fresh, tables, free, count, tokens = tr["before"]
        tables, free = tables.copy(), free.copy()
        want = R.kv_step(lens, fresh, tables, free, int(count[0]), 4, 6)
        seq, pos, slot, new_lens, starts, left = want
        got = tr["tables"]
        for a, b in zip(got, (seq, pos, slot, new_lens, starts, np.array([left]), tables, free)):
            assert np.array_equal(a, b)
        served = np.diff(starts) > 0
        assert np.array_equal(got[8], np.where(served, new_lens - 1, -1))
        rows = R.embed(np.where(served, tokens, -1), host(m.table.float()), 1.0)
        assert _same(tr["embed"][0], rows)                 # bf16 rows of a bf16 table
        delta, stream = tr["out"]
        xq, xs, logits = tr["head"]
        q0, s0, _, _ = BR.norm_quant(delta, host(m.norm), stream, 1e-6, 0, True)
        assert np.array_equal(xq, q0) and _same(xs, s0)
        if W is None:                                      # the head's weights, read back from its layout
            W = _unpack(m.head, 1003, 256, group)
        y, mag = R.q4_forward(xq, xs, *W, group)
        assert np.all(np.abs(logits - y) <= (256 // group + 8) * U * mag * (1 + 2.0 ** -8))
        temp, k, p = (host(m.settings[n]) for n in ("temperature", "top_k", "top_p"))
        for b in range(6):
            token, lp, d = R.sample_row(logits[b], u[b], temp[b], k[b], p[b])
            assert tr["tokens"][0][b] == token
            assert abs(tr["tokens"][1][b] - lp) <= 2.0 ** -22 * (1 + d) + 2.0 ** -24 * abs(lp)


def _unpack(head, n, K, group):
    """Quantized weights and scales of a packed head, element by element."""
    import torch
    codes, scales = host(head[0]), host(head[1].view(torch.int16)).view(np.uint16)
    NB, nt = -(-K // 128), -(-n // 16)
    codes, scales = codes.reshape(nt, NB, 64, 4, 4), scales.reshape(nt, NB, 4, 128 // group, 4)
    q, s = np.zeros((nt * 16, NB * 128), np.int8), np.zeros((nt * 16, NB * 128 // group), np.uint16)
    for l in range(64):
        h = l // 16
        for w in range(4):
            c = 32 * w + 8 * h if group == 32 else 64 * (w // 2) + 16 * h + 8 * (w % 2)
            for j in range(4):
                v = codes[:, :, l, w, j].astype(np.int16)
                for nib, at in ((v & 15, c + j), (v >> 4, c + 4 + j)):
                    q[l % 16::16, at::128] = (nib ^ 8) - 8
    for h in range(4):
        for i in range(128 // group):
            for r in range(4):
                s[4 * h + r::16, i::128 // group] = scales[:, :, h, i, r]
    s = (s.astype(np.uint32) << 16).view(np.float32)
    return q[:n, :K], s[:n, :K // group]


def test_steps_as_a_graph():
    """Replays equal eager steps: tokens, log probabilities, lengths and tables."""
    import torch
    runs = []
    for graphed in (False, True):
        m, g = _model(7)
        torch.cuda.synchronize()
        if graphed:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                m.step()
        out = []
        for t in range(10):
            m.fresh.copy_(dev(np.array(FRESH[t % len(FRESH)], np.int32)))
            m.u.copy_(dev(g.random(6)))
            if graphed:
                graph.replay()
            else:
                m.step()
            torch.cuda.synchronize()
            out.append([host(x).copy() for x in (m.tokens, m.logprob, m.lens, m.tables, m.free, m.rows.count)])
        runs.append(out)
    for x, y in zip(*runs):
        assert all(np.array_equal(a, b) for a, b in zip(x, y))


@pytest.mark.parametrize("accum", [False, True])
def test_training_half(accum):
    import torch

    import model as E
    g = rng(11)
    T, V, K, n, scale = 96, 40, 256, 320, 16.0
    table, w, W = (g.standard_normal(s).astype(np.float32) for s in ((V, K), K, (n, K)))
    w, W = 1 + np.float32(0.1) * w, W * np.float32(0.02)
    ids = np.minimum((V + 1.0) ** g.random(T) - 1, V - 1).astype(np.int32)
    ids[5] = -1
    dy = torch.from_numpy((g.standard_normal((T, n)) * 2.0 ** -10).astype(np.float32)).bfloat16().cuda()
    into = (g.standard_normal((V, K)) * 2.0 ** -10).astype(np.float32) if accum else None
    r = E.train_embedding(dev(ids), dev(table), dev(w), dev(W), dy, scale, dev(into) if accum else None)
    x = R.embed(ids, table, scale)
    assert _same(host(r["x"]), x)
    q0, s0, h0, r0 = BR.norm_quant(x, w)
    assert np.array_equal(host(r["xq"]), q0) and _same(host(r["scale"]), s0) and _same(host(r["rstd"]), r0)
    dh0, _ = BR.norm_grad(host(r["dn"]), h0, r0, w)
    dx = host(r["dx"])
    assert np.linalg.norm(dx - dh0) <= 2.0 ** -20 * np.linalg.norm(dh0)
    want, mag, count = R.embed_grad(dx, ids, V, scale, into)
    assert np.all(np.abs(host(r["dtable"]) - want) <= (count[:, None] + 1) * U * mag * (1 + 2.0 ** -8))
    # against differences: of sum(norm(embed(table)) * dn), the quantizer passed straight through
    ok = ids >= 0
    dn = host(r["dn"]).astype(np.float64)[ok]
    f = lambda t: (BR.norm_rows(t[ids[ok]] * scale, w.astype(np.float64), 1e-6) * dn).sum()  # noqa: E731
    full = host(r["dtable"]).astype(np.float64) - (into if accum else 0)
    for _ in range(6):
        v = g.standard_normal((V, K))
        e = 1e-5
        slope = (f(table + e * v) - f(table - e * v)) / (2 * e)
        # second differences are O(e^2); fp32 gradients carry (K + tokens) roundings of their terms
        assert abs(slope - (full * v).sum()) <= 1e-6 * (np.abs(full) * np.abs(v)).sum() + 1e-9


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_prompts_by_rows_of_a_step(kv):
    """Prompts of several tokens and single tokens in one step: kv_step's rows lead rope_append, its lengths and
    tables PagedAttn; its slots are where the keys went.  A request whose pages do not suffice adds nothing."""
    import torch
    g = rng(13)
    B, page, per, Hq, Hk, D, T = 5, 4, 6, 4, 2, 64, 40
    cached = np.array([0, 7, 9, 0, 3], np.int32)
    fresh = np.array([11, 1, 6, 20, 1], np.int32)
    tables = np.full((B, per), -1, np.int32)
    pool = g.permutation(17).astype(np.int32)
    n = 0
    for b in range(B):
        k = -(-int(cached[b]) // page)
        tables[b, :k] = pool[n:n + k]
        n += k
    free = np.concatenate((pool[n:], np.zeros(n, np.int32)))
    count = 17 - n - 5                                      # too few for the fourth request, which wants five
    kc, vc = (torch.randn(17, Hk, page, D, device="cuda") for _ in range(2))
    ks = vs = None
    if kv == "bf16":
        kc, vc = kc.bfloat16(), vc.bfloat16()
    else:
        kc, vc = ((c * 40).clamp(-127, 127).to(torch.int8) for c in (kc, vc))
        ks, vs = (0.01 + 0.01 * torch.rand(17, Hk, page, device="cuda") for _ in range(2))
    td, fd = dev(tables), dev(free)
    r = S.kv_step(dev(cached), dev(fresh), td, fd, dev(np.array([count], np.int32)), page, T)
    want = R.kv_step(cached, fresh, tables, free, count, page, T)
    assert np.array_equal(host(r.seq), want[0]) and want[3].tolist() == [11, 8, 15, 0, 4]
    q, k, v = (torch.randn(T, h, D, device="cuda") for h in (Hq, Hk, Hk))
    table = S.rope_table(per * page, *S.rope_frequencies(D))
    qr = S.rope_append(q, k, v, r.pos, table, kc, vc, td, seq=r.seq, k_scale=ks, v_scale=vs)
    rows = int(host(r.starts)[-1])
    kr = BR.rope(host(k), want[1], host(table))
    flat = host(kc.float()).transpose(0, 2, 1, 3).reshape(-1, Hk, D)
    for t in range(rows):
        if kv == "bf16":
            assert _same(flat[want[2][t]], BR.bf16_round(kr[t]))
        else:
            assert np.array_equal(flat[want[2][t]], O.act_quant(kr[t])[0])
    last = r.starts[1:].long() - 1                          # each request's newest token (those that wait: any)
    attn = S.PagedAttn(B, Hq, Hk, D, page, per * page)
    out = attn(qr[last.clamp(min=0)].contiguous(), kc, vc, td, r.lens, k_scale=ks, v_scale=vs)
    args = [host(x.float()) for x in (qr[last.clamp(min=0)], kc, vc)]
    scales = {} if kv == "bf16" else dict(ks=host(ks), vs=host(vs))
    ref, _, mag, smag = BR.paged_attn(*args, host(td), host(r.lens), D ** -0.5, **scales)
    e = ((D + 6) * U * smag + 4 * U + 2.0 ** -17 + 24 * U)[..., None]
    assert np.all(np.abs(host(out) - ref) <= 2 * e * mag + 1e-30)
    assert not host(out)[3].any()                           # nothing cached


@pytest.mark.parametrize("graphed", [False, True])
def test_a_request_that_waits_keeps_its_token(graphed):
    """A step leaves a request's token and log probability alone where it finds no page, adds nothing or has ended, and
    puts the draw from the request's logits there where it was served."""
    import torch
    m, g = _model(3, pages=9)
    step, waited = m.step, 0
    if graphed:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            m.step()
        step = graph.replay
    m.logprob.copy_(dev(np.arange(-6, 0, dtype=np.float32)))
    for t in range(16):
        fresh = np.array(FRESH[t % len(FRESH)], np.int32)
        m.fresh.copy_(dev(fresh))
        m.u.copy_(dev(g.random(6)))
        tokens, logprob = host(m.tokens).copy(), host(m.logprob).copy()
        step()
        served = np.diff(host(m.rows.starts)) > 0
        got = host(m.tokens)
        assert np.array_equal(got[~served], tokens[~served]) and _same(host(m.logprob)[~served], logprob[~served]), t
        logits = host(m.logits)
        for b in np.nonzero(served)[0]:
            want, lp, d = R.sample_row(logits[b], float(m.u[b]), float(m.settings["temperature"][b]),
                                       int(m.settings["top_k"][b]), float(m.settings["top_p"][b]))
            assert got[b] == want and abs(host(m.logprob)[b] - lp) <= 2.0 ** -22 * (1 + d) + 2.0 ** -24 * abs(
                lp), (t, b)
        waited += int((~served & (fresh > 0)).sum())
    assert waited == 25                                    # for a page, not by the caller's wish


def test_requests_as_long_as_their_pages():
    """A longest length inside a page: the pages' last positions have rows in the rotary table too, and a request is
    served up to the end of its table's row."""
    import model as E
    m = E.Model(3, layers=1, vocab=500, hidden=256, heads=4, kv_heads=2, D=64, ffn=320, page=8, max_len=17, seed=5)
    g = rng(5)
    for t in range(26):
        m.u.copy_(dev(g.random(3)))
        m.step()
        assert host(m.lens).tolist() == [min(t + 1, 24)] * 3
        assert (host(m.tokens) >= 0).all() and np.isfinite(host(m.logprob)).all() and np.isfinite(host(m.logits)).all(), t
