"""What the operators between the projections accept and refuse of strides and overlaps (CPU only): the C ABI
answers before it touches the HIP runtime (fake, never dereferenced device addresses; calls of no tokens
return before a launch)."""
import ctypes

import pytest

from sparsity_amd import block as K

P = 1 << 40                                # fake, 256-byte aligned; buffers 16 GiB apart
SLOT = 16 << 30
EINVAL = -22


def _desc(x, y=None, **kw):
    a = dict(x=x, y=y, x_tok=2048, x_head=128, y_tok=2048, y_head=128, heads=4)
    a.update(kw)
    return K.BlRopeDesc(*a.values())


def _kv(**kw):
    a = dict(k=P + 30 * SLOT, v=P + 40 * SLOT, ks=P + 50 * SLOT, vs=P + 51 * SLOT, page=16 * 4 * 128, head=16 * 128,
             tok=128, pages=100, page_size=16, heads=4, dim=128, dtype=2)
    a.update(kw)
    return K.BlKvCache(*a.values())


def _append(q=None, k=None, v=None, **kw):
    arr = (K.BlRopeDesc * 3)(q or _desc(P, P + 10 * SLOT), k or _desc(P + SLOT), v or _desc(P + 2 * SLOT))
    a = dict(T=0, R=128, inter=0, xd=0, qd=0, pos=P + 20 * SLOT, seq=None, blocks=P + 21 * SLOT, seqs=4, per=8,
             table=P + 22 * SLOT, n=64, kv=_kv())
    a.update(kw)
    return K.bitlinear_rope_append(arr, *a.values(), None)


@pytest.mark.parametrize("kw", [dict(pages=1, page=12345), dict(pages=1, page=-7), dict(heads=1, head=3),
                                dict(page_size=1, tok=5, head=128, page=512),
                                dict(pages=1, heads=1, page_size=1, page=1, head=2, tok=3)])
def test_cache_strides_of_axes_of_one(kw):
    heads = kw.get("heads", 4)
    k = _desc(P + SLOT, heads=heads), _desc(P + 2 * SLOT, heads=heads)
    assert _append(k=k[0], v=k[1], kv=_kv(**kw)) == 0
    st, plan = K.bitlinear_paged_attn_plan(0, 4, heads, 128, 10, 0)
    assert st == 0
    assert K.bitlinear_paged_attn(ctypes.byref(plan), None, 0, 0, 0, 1.0, _kv(**kw), None, 1, None, None, None, None,
                                  0, None) == 0
