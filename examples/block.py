#!/usr/bin/env python3
"""A ternary decoder block on the library: decode steps over a paged cache, and a training step of its
attention input.

``DecodeBlock`` holds one block's packed 2:4 weights, its buffers and its cache; a step is

    norm_quant (+ residual) -> q, k, v projections -> rope_append -> PagedAttn -> act_quant -> o
    projection -> norm_quant (+ residual) -> gate, up projections -> squared ReLU gate -> norm_quant
    -> down projection

with every projection's independent parts in one grouped launch.  ``train_attention_input`` runs the
norm, the projections and the rotary positions forward and backward.  Weights are random:

    python examples/block.py                 # 16 sequences, prompts of 24 to 99 tokens, 32 steps
    python examples/block.py --kv int8
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparsity_amd as S  # noqa: E402


class DecodeBlock:
    def __init__(self, seqs, hidden=2560, heads=20, kv_heads=5, D=128, ffn=6912, page=16, max_len=512,
                 kv="bf16", seed=0):
        dev = torch.device("cuda")
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.seqs, self.heads, self.kv_heads, self.D, self.max_len = seqs, heads, kv_heads, D, max_len

        def packed(n, K):
            W = torch.randn(n, K, generator=g, device=dev) * 0.02
            return dict(zip(("codes", "meta", "gamma"), S.pack(W)), K=K, n=n)

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=dev)

        def project(layers, rows):   # the projections of one input, its int8 rows and their scales
            K = layers[0]["K"]
            xq, scale = empty(rows, K, dtype=torch.int8), empty(max(rows, 4))[:rows]
            ys = [empty(rows, w["n"]) for w in layers]
            group = S.FwdGroup([dict(w, xq=xq, scale=scale, y=y) for w, y in zip(layers, ys)])
            return xq, scale, ys, group

        self.w1, self.w2 = (1 + 0.1 * torch.randn(hidden, generator=g, device=dev) for _ in range(2))
        self.w3 = 1 + 0.1 * torch.randn(ffn, generator=g, device=dev)
        self.qkv = project([packed(heads * D, hidden), packed(kv_heads * D, hidden),
                            packed(kv_heads * D, hidden)], seqs)
        self.o = project([packed(hidden, heads * D)], seqs)
        self.gate_up = project([packed(ffn, hidden), packed(ffn, hidden)], seqs)
        self.down = project([packed(hidden, ffn)], seqs)

        freq, mscale = S.rope_frequencies(D)
        self.table = S.rope_table(max_len, freq, mscale)
        per = -(-max_len // page)
        pages = seqs * per
        shape = (pages, kv_heads, page, D)
        dtype = torch.int8 if kv == "int8" else torch.bfloat16
        self.k_cache, self.v_cache = torch.zeros(shape, dtype=dtype, device=dev), torch.zeros(
            shape, dtype=dtype, device=dev)
        self.scales = {}
        if kv == "int8":
            self.scales = {n: torch.zeros(shape[:3], device=dev) for n in ("k_scale", "v_scale")}
        self.blocks = torch.randperm(pages, generator=g, device=dev).int().view(seqs, per)
        self.attn = S.PagedAttn(seqs, heads, kv_heads, D, page, max_len)
        self.stream = empty(seqs, hidden, dtype=torch.bfloat16)   # the residual stream
        self.q = empty(seqs, heads, D, dtype=torch.bfloat16)
        self.mixed = empty(seqs, heads, D, dtype=torch.bfloat16)

    def step(self, delta, pos, lens, trace=None):
        """One token per sequence: adds delta (fp32 [seqs][hidden], the previous block's output) to the
        residual stream and returns this block's output; pos and lens (= pos + 1) are int32 [seqs]."""
        keep = (lambda n, *t: None) if trace is None else (lambda n, *t: trace.append(
            (n, [x.clone() for x in t])))
        keep("in", delta, self.stream)
        xq, scale, (q, k, v), group = self.qkv
        S.norm_quant(delta, self.w1, self.stream, out=(xq, scale, self.stream, None))
        group()
        keep("qkv", xq, scale, self.stream, q, k, v)
        S.rope_append(q.view(self.seqs, self.heads, self.D), k.view(self.seqs, self.kv_heads, self.D),
                      v.view(self.seqs, self.kv_heads, self.D), pos, self.table, self.k_cache,
                      self.v_cache, self.blocks, out=self.q, **self.scales)
        self.attn(self.q, self.k_cache, self.v_cache, self.blocks, lens, out=self.mixed, **self.scales)
        keep("attn", self.q, self.mixed)
        xq, scale, (y,), group = self.o
        S.act_quant(self.mixed.view(self.seqs, -1), out=(xq, scale))
        group()
        keep("o", xq, scale, y)
        xq, scale, (gate, up), group = self.gate_up
        S.norm_quant(y, self.w2, self.stream, out=(xq, scale, self.stream, None))
        group()
        keep("gate_up", xq, scale, self.stream, gate, up)
        inner = torch.relu(gate).square_().mul_(up)
        xq, scale, (y,), group = self.down
        S.norm_quant(inner, self.w3, out=(xq, scale, None, None))
        group()
        keep("down", inner, xq, scale, y)
        return y


def train_attention_input(T=512, hidden=2560, heads=20, D=128, seed=0):
    """Norm, one projection and rotary positions of T tokens, forward and backward; returns a dict of
    everything that was computed."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    W, w = rnd(heads * D, hidden) * 0.02, 1 + 0.1 * rnd(hidden)
    x, res = rnd(T, hidden), rnd(T, hidden).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    table = S.rope_table(T, *S.rope_frequencies(D))
    packed = S.pack(W)
    # forward
    xq, scale, h, rstd = S.norm_quant(x, w, res, want_rstd=True)
    y = S.fwd(xq, scale, hidden, *packed, heads * D)
    q, = S.rope([y.view(T, heads, D)], pos, table, dtype=torch.bfloat16)
    # backward, from the gradients of q and of the residual stream behind this point
    dq, dstream = (rnd(T, heads, D) * 2.0 ** -10).bfloat16(), (rnd(T, hidden) * 2.0 ** -10).bfloat16()
    dy, = S.rope([dq], pos, table, inverse=True)
    dn, dW = S.bwd(dy.view(T, -1), xq, scale, hidden, *packed, heads * D)
    dh, dw = S.norm_quant_bwd(dn, h, rstd, w, dstream)
    return dict(W=W, w=w, x=x, res=res, pos=pos, table=table, packed=packed, xq=xq, scale=scale, h=h,
                rstd=rstd, y=y, q=q, dq=dq, dstream=dstream, dy=dy, dn=dn, dW=dW, dh=dh, dw=dw)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=16)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--kv", choices=("bf16", "int8"), default="bf16")
    a = ap.parse_args()
    block = DecodeBlock(a.seqs, kv=a.kv)
    # prompts of different lengths, a token at a time; a sequence whose prompt has not begun is padding
    prompt = torch.arange(a.seqs, device="cuda", dtype=torch.int32) * 5 + 24
    block.stream.normal_()
    delta = torch.zeros(a.seqs, 2560, device="cuda")
    longest = int(prompt.max())
    for t in range(longest):
        pos = t - (longest - prompt)
        delta = block.step(delta, pos, (pos + 1).clamp_(min=0))
        block.stream.normal_()
    torch.cuda.synchronize()
    began = time.perf_counter()
    for t in range(a.steps):
        pos = prompt + t
        delta = block.step(delta, pos, pos + 1)
    torch.cuda.synchronize()
    took = (time.perf_counter() - began) / a.steps
    assert bool(torch.isfinite(delta).all())
    # the same step as a graph: positions and lengths are read from their buffers at each replay
    pos, lens = prompt + a.steps, prompt + a.steps + 1
    delta, graph = delta.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        delta.copy_(block.step(delta, pos, lens))
    torch.cuda.synchronize()
    began = time.perf_counter()
    for t in range(a.steps):
        graph.replay()
        pos += 1
        lens += 1
    torch.cuda.synchronize()
    replayed = (time.perf_counter() - began) / a.steps
    print(f"decode: {a.seqs} sequences, {a.steps} steps, {took * 1e6:.0f} us per step of one block "
          f"({replayed * 1e6:.0f} us as a graph), {a.kv} cache")
    out = train_attention_input()
    assert bool(torch.isfinite(out["dh"].float()).all())
    print(f"training: dh {tuple(out['dh'].shape)}, dW {tuple(out['dW'].shape)}, dw {tuple(out['dw'].shape)}")


if __name__ == "__main__":
    main()
