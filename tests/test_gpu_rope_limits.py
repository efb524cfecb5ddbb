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
