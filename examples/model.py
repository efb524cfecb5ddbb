#!/usr/bin/env python3
"""A ternary decoder from token ids to token ids: requests come and go, every step adds a token to each.

``Model`` puts the ends around ``block.py``'s decoder blocks.  A step is

    kv_step (pages for the new tokens, ended requests' pages back) -> embed -> the blocks -> norm_quant
    -> q4_fwd (an output head in 4 bits) -> sample

all on the GPU, so that it can be captured: the next step's token ids are where this one left them.
``train_embedding`` runs the embedding's training half, forward and backward.  Weights are random:

    python examples/model.py                 # 16 requests at a time, 2 blocks, 48 steps
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import sparsity_amd as S  # noqa: E402
from block import DecodeBlock  # noqa: E402


class Model:
    def __init__(self, seqs, layers=2, vocab=32000, hidden=2560, heads=20, kv_heads=5, D=128, ffn=6912, page=16,
                 max_len=512, pages=None, kv="bf16", group=64, seed=0):
        per = -(-max_len // page)
        max_len = per * page                                   # kv_step fills pages to their ends
        if pages is None:
            pages = seqs * per
        if not 0 <= pages <= seqs * per:
            raise ValueError(f"pages: the layers' caches have {seqs * per}, got {pages}")
        dev = torch.device("cuda")
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.seqs, self.page, self.vocab, self.hidden, self.group = seqs, page, vocab, hidden, group
        self.layers = [DecodeBlock(seqs, hidden, heads, kv_heads, D, ffn, page, max_len, kv, seed + 1 + i)
                       for i in range(layers)]

        def empty(*shape, dtype=torch.int32):
            return torch.empty(shape, dtype=dtype, device=dev)

        # one table of pages for all layers, whose caches are alike; all pages are free at first
        self.tables = torch.full((seqs, per), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(pages, dtype=torch.int32, device=dev)
        self.lens, self.fresh = torch.zeros(seqs, dtype=torch.int32, device=dev), torch.ones(seqs, dtype=torch.int32,
                                                                                         device=dev)
        self.rows = S.KvStep(empty(seqs), empty(seqs), empty(seqs, dtype=torch.int64), self.lens, empty(seqs + 1),
                             torch.tensor([pages], dtype=torch.int32, device=dev))
        self.stream = empty(seqs, hidden, dtype=torch.bfloat16)
        for b in self.layers:
            b.blocks, b.stream = self.tables, self.stream
        self.none = torch.zeros(seqs, hidden, device=dev)
        self.table = torch.randn(vocab, hidden, generator=g, device=dev).bfloat16()
        self.norm = 1 + 0.1 * torch.randn(hidden, generator=g, device=dev)
        self.head = S.q4_pack(torch.randn(vocab, hidden, generator=g, device=dev) * 0.02, group)
        self.xq, self.scale = empty(seqs, hidden, dtype=torch.int8), empty(seqs, dtype=torch.float32)
        self.logits = empty(seqs, vocab, dtype=torch.float32)
        # each request's token, settings and next random number; what a step draws, for rows without a request too
        self.tokens = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.logprob = torch.zeros(seqs, dtype=torch.float32, device=dev)
        self.drawn = empty(seqs), empty(seqs, dtype=torch.float32)
        self.u = torch.zeros(seqs, dtype=torch.float64, device=dev)
        self.settings = dict(temperature=torch.full((seqs,), 0.8, device=dev),
                             top_k=torch.full((seqs,), 50, dtype=torch.int32, device=dev),
                             top_p=torch.full((seqs,), 0.95, device=dev), min_p=torch.zeros(seqs, device=dev))
        self.ws = empty(S.bitlinear_sample_workspace_bytes(seqs, vocab)[1], dtype=torch.uint8)

    def step(self, trace=None):
        """One token per request, from self.tokens and to self.tokens.  fresh is 1 for a request that goes on, -1 for
        one that has ended (its place begins anew at length 0 with the next step's 1, from the token that the caller
        puts there), 0 for an empty place.  A request that kv_step does not serve keeps its token and waits."""
        keep = (lambda n, *t: None) if trace is None else (lambda n, *t: trace.append(
            (n, [x.clone() for x in t])))
        keep("before", self.lens, self.fresh, self.tables, self.free, self.rows.count, self.tokens)
        S.kv_step(self.lens, self.fresh, self.tables, self.free, self.rows.count, self.page, self.seqs, out=self.rows)
        served = self.rows.starts.diff() > 0
        pos = torch.where(served, self.lens - 1, -1)           # rows in the order of requests: -1 adds nothing
        keep("tables", *self.rows, self.tables, self.free, pos)
        S.embed(torch.where(served, self.tokens, -1), self.table, out=self.stream)
        keep("embed", self.stream)
        delta = self.none
        for b in self.layers:
            delta = b.step(delta, pos, self.lens)
        keep("out", delta, self.stream)
        S.norm_quant(delta, self.norm, self.stream, out=(self.xq, self.scale, self.stream, None))
        S.q4_fwd(self.xq, self.scale, self.hidden, *self.head, self.vocab, self.group, out=self.logits)
        keep("head", self.xq, self.scale, self.logits)
        S.sample(self.logits, self.u, **self.settings, out=self.drawn, ws=self.ws)
        keep("tokens", *self.drawn)
        for mine, drawn in zip((self.tokens, self.logprob), self.drawn):
            mine.copy_(torch.where(served, drawn, mine))
        return self.tokens


def train_embedding(ids, table, weight, W, dy, scale=1.0, dtable=None):
    """Embedding rows of ids (int32 [T]) from an fp32 table [V][K], norm and one projection, and the gradients that
    come back from dy (bf16 [T][n]) with the residual stream's own share: a dict of everything that was computed.
    dtable, if given, is added to (a tied output head's gradient)."""
    V, K = table.shape
    packed = S.pack(W)
    x = S.embed(ids, table, scale=scale)
    xq, xs, _, rstd = S.norm_quant(x, weight, want_rstd=True)
    y = S.fwd(xq, xs, K, *packed, W.shape[0])
    dn, dW = S.bwd(dy, xq, xs, K, *packed, W.shape[0])
    dx, dw = S.norm_quant_bwd(dn, x, rstd, weight)
    dt = S.embed_bwd(dx, ids, V, scale=scale, accumulate=dtable is not None, out=dtable)
    return dict(packed=packed, x=x, xq=xq, scale=xs, rstd=rstd, y=y, dn=dn, dW=dW, dx=dx, dw=dw, dtable=dt)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=16)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--steps", type=int, default=48)
    a = ap.parse_args()
    m = Model(a.seqs, a.layers)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    m.tokens.random_(0, m.vocab, generator=g)
    for _ in range(3):
        m.u.uniform_(generator=g)
        m.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    began = time.perf_counter()
    for t in range(a.steps):
        m.u.uniform_(generator=g)
        place = t // 16 % a.seqs
        if t % 16 == 15:                   # one request ends, another takes its place with the step after
            m.fresh[place] = -1
        graph.replay()
        if t % 16 == 15:
            m.fresh[place] = 1
            m.tokens[place:place + 1].random_(0, m.vocab, generator=g)
    torch.cuda.synchronize()
    took = (time.perf_counter() - began) / a.steps
    assert bool(((m.tokens >= 0) & (m.tokens < m.vocab)).all()) and bool(torch.isfinite(m.logprob).all())
    print(f"{a.seqs} requests, {a.layers} blocks, {m.vocab} tokens: {took * 1e6:.0f} us per step as a graph, lengths "
          f"{int(m.lens.min())} to {int(m.lens.max())}, {int(m.rows.count)} pages left")
    T, V, K, n = 512, 4000, 2560, 2560
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    out = train_embedding(ids, rnd(V, K), 1 + 0.1 * rnd(K), rnd(n, K) * 0.02, rnd(T, n).bfloat16())
    assert bool(torch.isfinite(out["dtable"]).all())
    print(f"training: x {tuple(out['x'].shape)}, dtable {tuple(out['dtable'].shape)}")


if __name__ == "__main__":
    main()
