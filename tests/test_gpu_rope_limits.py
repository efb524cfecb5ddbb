"""Rotary positions and the append where buffers meet: in place on rows of any alignment, and slices of one
buffer beside each other.  Results equal the definition to the bit."""
import numpy as np
import pytest

import oracle.block_ref as R
from parity_util import dev, f32_bits, host
from synth import rng

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")


def _same(a, b):
    return np.array_equal(f32_bits(np.ascontiguousarray(a)), f32_bits(np.ascontiguousarray(b)))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,Rt,off", [(1, 20, 5, 128, 128, 1), (33, 25, 5, 80, 78, 2), (300, 9, 3, 256, 254, 0),
                                              (1100, 32, 8, 64, 22, 1), (5, 7, 1, 48, 48, 3)])
def test_append_in_place_reads_a_pair_before_it_writes(inter, bf16, T, Hq, Hk, D, Rt, off):
    """Queries rotated in place on the path that reads the other half of each pair from memory."""
    import torch
    g = rng(T + D)
    dt = torch.bfloat16 if bf16 else torch.float32
    W = (Hq + 2 * Hk) * D + 5
    x = g.standard_normal((T, W)).astype(np.float32)
    if bf16:
        x = R.bf16_round(x)
    rows = torch.zeros(T * W + off, dtype=dt, device="cuda")[off:].view(T, W)
    rows.copy_(dev(x))
    cut = lambda a, h: rows[:, a:a + h * D].unflatten(1, (h, D))
    q, k, v = cut(0, Hq), cut(Hq * D, Hk), cut((Hq + Hk) * D, Hk)
    table = R.rope_table(S.rope_frequencies(Rt)[0], T + 3)
    pos = g.permutation(T + 3)[:T].astype(np.int32)
    ps = 16
    per = -(-(T + 3) // ps)
    kc, vc = (torch.zeros(per, Hk, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    blocks = np.arange(per, dtype=np.int32)[None]
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    out = S.rope_append(q, k, v, dev(pos), dev(table), kc, vc, dev(blocks), seq, interleaved=inter, out=q)
    cast = R.bf16_round if bf16 else (lambda a: a)
    qkv = x[:, :(Hq + 2 * Hk) * D].reshape(T, Hq + 2 * Hk, D)
    turned = R.rope(qkv[:, :Hq + Hk], pos, table, inter)
    assert _same(host(out.float()), cast(turned[:, :Hq]))
    got = host(rows.float())
    assert _same(got[:, :Hq * D], cast(turned[:, :Hq]).reshape(T, -1)) and _same(got[:, Hq * D:], x[:, Hq * D:])
    flat = lambda c: host(c.float()).transpose(0, 2, 1, 3).reshape(per * ps, Hk, D)[pos]
    assert _same(flat(kc), R.bf16_round(turned[:, Hq:])) and _same(flat(vc), R.bf16_round(qkv[:, Hq + Hk:]))


def test_slices_of_one_buffer_do_not_overlap():
    """Slices beside each other in rows, heads and pages, in place and from one slice into the next one's
    neighbour, are not taken for overlaps."""
    import torch
    g = rng(71)
    T, D = 40, 32
    table = R.rope_table(S.rope_frequencies(D)[0], 64)
    pos = g.permutation(64)[:T].astype(np.int32)
    x = g.standard_normal((T, 12, D)).astype(np.float32)
    want = R.rope(x, pos, table)
    b = dev(x)                                                            # heads 0..3, 4..5 in place
    S.rope([b[:, :4], b[:, 4:6]], dev(pos), dev(table), outs=[b[:, :4], b[:, 4:6]])
    assert _same(host(b)[:, :6], want[:, :6]) and _same(host(b)[:, 6:], x[:, 6:])
    b = dev(x)                                                            # into the same row's other heads
    S.rope([b[:, :3], b[:, 3:6]], dev(pos), dev(table), outs=[b[:, 6:9], b[:, 9:]])
    assert _same(host(b)[:, 6:], want[:, :6]) and _same(host(b)[:, :6], x[:, :6])
    b = dev(x)                                                            # even heads into odd ones
    S.rope([b[:, 0::2]], dev(pos), dev(table), outs=[b[:, 1::2]])
    assert _same(host(b)[:, 1::2], want[:, 0::2]) and _same(host(b)[:, 0::2], x[:, 0::2])
    b = dev(x.transpose(1, 0, 2))                                         # head-major: halves of a buffer
    v = b.transpose(0, 1)
    S.rope([v[:, :6]], dev(pos), dev(table), outs=[v[:, 6:]])
    assert _same(host(v.contiguous())[:, 6:], want[:, :6])
    b = dev(x)                                                            # unlike strides: odd tokens, one head
    S.rope([b[0::2]], dev(pos[0::2]), dev(table), outs=[b[1::2]])
    assert _same(host(b)[1::2], R.rope(x[0::2], pos[0::2], table))
    # keys and values of one cache buffer: by page, by head and by row
    Hk, ps, seqs = 2, 8, 5
    blocks = np.arange(seqs * 8, dtype=np.int32).reshape(seqs, 8)
    seq = (np.arange(T) % seqs).astype(np.int32)
    where = (np.arange(T) // seqs).astype(np.int32)
    kr = R.bf16_round(R.rope(x[:, 4:6], where, table))
    vr = R.bf16_round(x[:, 6:8])
    q = R.rope(x[:, :4], where, table)
    for shape, cut in (((40, 2, Hk, ps, D), lambda c, i: c[:, i]), ((40, Hk, 2, ps, D), lambda c, i: c[:, :, i]),
                       ((40, Hk, ps, 2, D), lambda c, i: c[:, :, :, i]),
                       ((40, ps, Hk, 2, D), lambda c, i: c[:, :, :, i].transpose(1, 2))):
        c = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        kc, vc = cut(c, 0), cut(c, 1)
        b = dev(x)
        out = S.rope_append(b[:, :4], b[:, 4:6], b[:, 6:8], dev(where), dev(table), kc, vc, dev(blocks), dev(seq),
                            out=b[:, 8:])
        assert _same(host(out.contiguous()), q)
        pg, off = blocks[seq, where // ps], where % ps
        for got, w in ((kc, kr), (vc, vr)):
            assert _same(host(got.float())[pg, :, off], w)
