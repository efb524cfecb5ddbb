"""What the operators between the projections accept and refuse of strides and overlaps, and the device they
are enqueued on (CPU only): the C ABI answers before it touches the HIP runtime (fake, never dereferenced
device addresses; calls of no tokens return before a launch)."""
import contextlib
import ctypes

import pytest
import torch

import sparsity_amd as S
from sparsity_amd import block as K
from test_block_abi import BF, F32, I8, I32, Strided

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


def _rope(*descs, **kw):
    a = dict(T=4, D=128, R=128, inter=0, inv=0, xd=0, yd=0, pos=P + 20 * SLOT, table=P + 21 * SLOT, n=64)
    a.update(kw)
    return K.bitlinear_rope((K.BlRopeDesc * len(descs))(*descs), *a.values(), None)


ROW = 128 * 4                              # bytes of a head


@pytest.mark.parametrize("descs,kw", [
    ([_desc(P, P + ROW)], {}),                                            # shifted over itself by a head
    ([_desc(P, P + 4 * ROW - 4, x_tok=512, y_tok=512)], {}),              # by a token less an element
    ([_desc(P, P + SLOT), _desc(P + SLOT, P + 3 * SLOT)], {}),            # one tensor's output is another's input
    ([_desc(P, P + SLOT), _desc(P + 2 * SLOT, P)], {}),
    ([_desc(P, P + SLOT), _desc(P + 2 * SLOT, P + SLOT)], {}),            # two outputs in one place
    ([_desc(P, P), _desc(P, P)], {}),                                     # one tensor in place twice
    ([_desc(P, P), _desc(P + 3 * ROW, P + SLOT)], {}),                    # slices of a fused row that share a head
    ([_desc(P, P), _desc(P + 4 * ROW, P + 4 * ROW), _desc(P + 8 * ROW, P + 7 * ROW + 4)], {}),
    ([_desc(P, P + SLOT, y_head=256), _desc(P + SLOT + 3 * ROW - 4, P + 3 * SLOT, x_head=256)], {}),   # every other head
    ([_desc(P, P + SLOT, x_tok=512), _desc(P + SLOT + 3 * 8192 + 100, P + 3 * SLOT, x_tok=640)], {}),  # unlike strides
    ([_desc(P, P + 20 * SLOT - 64)], {}),                                 # over the positions
    ([_desc(P, P + 21 * SLOT + 64 * 512 - 16)], {}),                      # over the table's last entries
    ([_desc(P, P + SLOT), _desc(P + SLOT + 4, P + 3 * SLOT)], dict(xd=1, yd=0))])
def test_rope_refuses_overlaps(descs, kw):
    assert _rope(*descs, **kw) == EINVAL


KV = 100 * 16 * 4 * 128                    # bytes of an int8 cache, and four times those of its scales


@pytest.mark.parametrize("kw", [
    dict(q=_desc(P, P + SLOT)), dict(q=_desc(P, P + 2 * SLOT + ROW)), dict(q=_desc(P, P + ROW)),
    dict(q=_desc(P, P + 20 * SLOT)), dict(q=_desc(P, P + 21 * SLOT)), dict(q=_desc(P, P + 22 * SLOT)),
    dict(q=_desc(P, P + 30 * SLOT + KV - 64)), dict(q=_desc(P, P + 40 * SLOT)), dict(q=_desc(P, P + 51 * SLOT + 64)),
    dict(seq=P + 10 * SLOT), dict(k=_desc(P + 30 * SLOT + 512)), dict(v=_desc(P + 40 * SLOT)),
    dict(kv=_kv(v=P + 30 * SLOT)), dict(kv=_kv(v=P + 30 * SLOT + KV - 128)), dict(kv=_kv(vs=P + 50 * SLOT)),
    dict(kv=_kv(vs=P + 50 * SLOT + 100 * 64 * 4 - 4)), dict(kv=_kv(ks=P + 40 * SLOT + 256)),
    dict(kv=_kv(k=P + 20 * SLOT)), dict(kv=_kv(ks=P + 21 * SLOT)), dict(kv=_kv(v=P + 22 * SLOT + 64)),
    # keys and values side by side in rows or pages that are too short for both
    dict(kv=_kv(v=P + 30 * SLOT + 112, tok=256, head=4096, page=16384)),
    dict(kv=_kv(v=P + 30 * SLOT + 3 * 2048, page=2 * 8192, heads=4))])
def test_append_refuses_overlaps(kw):
    assert _append(T=4, **kw) == EINVAL


class Placed(Strided):
    def data_ptr(self):
        return P


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    """With another device current, a call makes its tensors' device current, takes that device's stream, and
    leaves the current device as it was."""
    now = [0]

    @contextlib.contextmanager
    def device(index):
        was, now[0] = now[0], index
        yield
        now[0] = was

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, now[0], args[-1]))
                return 0
            return call

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i if now[0] == i else None,
                        raising=False)
    plan = S.PagedAttn(4, 8, 2, 64, 16, 100, device="cpu")
    monkeypatch.setattr(K, "_lib", lambda: Lib())
    for index in (1, 0, 2):
        calls = []
        t = lambda shape, dtype: Placed(shape, dtype, device=torch.device("cuda", index))   # noqa: B023
        plan.ws = t(plan.plan.ws_bytes, torch.uint8)
        x, w, h, r = t((4, 256), F32), t(256, F32), t((4, 256), BF), t(4, F32)
        S.norm_quant(x, w, h, out=(t((4, 256), I8), r, h, r))
        S.norm_quant_bwd(x, h, r, w, h, out=(h, None))
        table, pos, blocks = t((50, 32, 2), F32), t(4, I32), t((4, 2), I32)
        S.rope_table(50, t(32, torch.float64), out=table)
        q, k, c = t((4, 8, 64), BF), t((4, 2, 64), BF), t((9, 2, 16, 64), BF)
        S.rope([q], pos, table, outs=[q])
        S.rope_append(q, k, k, pos, table, c, c, blocks, out=q)
        plan(q, c, c, blocks, pos, out=q)
        assert [n for n, _, _ in calls] == ["bitlinear_norm_quant", "bitlinear_norm_quant_bwd", "bitlinear_rope_table",
                                            "bitlinear_rope", "bitlinear_rope_append", "bitlinear_paged_attn"]
        assert all(d == index and s == 1000 + index for _, d, s in calls) and now == [0]
