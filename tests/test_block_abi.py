"""Refusals of the operators between the projections (CPU only): the C ABI rejects bad arguments
before it touches the HIP runtime (fake, never dereferenced device addresses are passed), and the
torch wrappers reject wrong tensors before anything reaches the C ABI."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.block_ref as R
import sparsity_amd as S
from sparsity_amd import block as K
from test_binding_checks import DEV, FakeT

P = 1 << 40                                # fake, 256-byte aligned; buffers 16 GiB apart
SLOT = 16 << 30
EINVAL, ENOTSUP, ENOSPC = -22, -95, -28


def _norm(**kw):
    a = dict(x=P, xd=0, res=P + SLOT, rd=1, w=P + 2 * SLOT, eps=1e-6, T=4, K=256, lift=0, h=P + 3 * SLOT,
             xq=P + 4 * SLOT, sc=P + 5 * SLOT, rstd=P + 6 * SLOT)
    a.update(kw)
    return K.bitlinear_norm_quant(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(xd=2), ENOTSUP), (dict(rd=7), ENOTSUP), (dict(K=252), EINVAL), (dict(K=0), EINVAL),
    (dict(K=32776), ENOTSUP), (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL), (dict(T=1 << 22), EINVAL),
    (dict(eps=0.0), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL), (dict(eps=math.inf), EINVAL),
    (dict(lift=4), EINVAL), (dict(lift=7), EINVAL), (dict(lift=6, K=256), EINVAL), (dict(lift=18), EINVAL),
    (dict(x=None), EINVAL), (dict(x=P + 8), EINVAL), (dict(xq=None), EINVAL), (dict(xq=P + 4 * SLOT + 4), EINVAL),
    (dict(sc=None), EINVAL), (dict(sc=P + 2), EINVAL), (dict(h=None), EINVAL), (dict(res=None), EINVAL),
    (dict(res=P + SLOT + 2), EINVAL), (dict(w=P + 4), EINVAL), (dict(rstd=P + 6 * SLOT + 1), EINVAL),
    (dict(h=P), EINVAL),                                    # over x of another type
    (dict(h=P + SLOT + 16), EINVAL),                        # shifted over the residual
    (dict(xq=P), EINVAL), (dict(xq=P + 2 * SLOT), EINVAL), (dict(sc=P + 4 * SLOT + 16), EINVAL),
    (dict(rstd=P + 5 * SLOT + 8), EINVAL), (dict(T=0, x=None, res=None, h=None, xq=None, sc=None), 0)])
def test_norm_quant_rejects(kw, want):
    assert _norm(**kw) == want


def _bwd(**kw):
    a = dict(dn=P, dd=0, h=P + SLOT, hd=1, rstd=P + 2 * SLOT, w=P + 3 * SLOT, dres=P + 4 * SLOT, dh=P + 5 * SLOT,
             gd=1, dw=P + 6 * SLOT, T=100000, K=256, ws=P + 7 * SLOT, wsb=1 << 30)
    a.update(kw)
    return K.bitlinear_norm_quant_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dd=2), ENOTSUP), (dict(hd=-1), ENOTSUP), (dict(gd=2), ENOTSUP), (dict(K=12), EINVAL),
    (dict(K=1 << 16), ENOTSUP), (dict(T=-2), EINVAL), (dict(dn=None), EINVAL), (dict(h=P + 2), EINVAL),
    (dict(rstd=None), EINVAL), (dict(dh=None), EINVAL), (dict(dres=P + 6), EINVAL), (dict(w=P + 4), EINVAL),
    (dict(dw=P + 8), EINVAL), (dict(ws=None), EINVAL), (dict(wsb=256 * 256 * 4 - 1), ENOSPC), (dict(wsb=0), ENOSPC),
    (dict(dh=P), EINVAL), (dict(dh=P + 4 * SLOT + 16), EINVAL), (dict(dh=P + SLOT), EINVAL),
    (dict(dw=P + 3 * SLOT), EINVAL), (dict(ws=P + 6 * SLOT), EINVAL), (dict(dw=P + 5 * SLOT), EINVAL),
    (dict(T=0, dw=None, dn=None, h=None), 0)])
def test_norm_grad_rejects(kw, want):
    assert _bwd(**kw) == want


def test_norm_grad_workspace():
    for T in (0, 1, 700):                                  # few rows: dw is summed by columns
        assert K.bitlinear_norm_quant_bwd_workspace_bytes(T, 3200) == (0, 0)
    st, most = K.bitlinear_norm_quant_bwd_workspace_bytes(1 << 20, 3200)
    assert st == 0 and most == 256 * 3200 * 4
    assert K.bitlinear_norm_quant_bwd_workspace_bytes(1, 100)[0] == EINVAL
    assert K.bitlinear_norm_quant_bwd_workspace_bytes(1, 32776)[0] == ENOTSUP


def _desc(i=0, **kw):
    a = dict(x=P + i * SLOT, y=P + (8 + i) * SLOT, x_tok=512, x_head=128, y_tok=512, y_head=128, heads=4)
    a.update(kw)
    return K.BlRopeDesc(*a.values())


def _rope(descs=None, **kw):
    descs = [_desc()] if descs is None else descs
    a = dict(T=4, D=128, R=128, inter=0, inv=0, xd=0, yd=1, pos=P + 20 * SLOT, table=P + 21 * SLOT, n=64)
    a.update(kw)
    return K.bitlinear_rope((K.BlRopeDesc * len(descs))(*descs), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(xd=2), ENOTSUP), (dict(yd=3), ENOTSUP), (dict(D=0), EINVAL), (dict(D=257), EINVAL), (dict(R=3), EINVAL),
    (dict(R=0), EINVAL), (dict(R=130), EINVAL), (dict(T=-1), EINVAL), (dict(T=1 << 22), EINVAL), (dict(n=-1), EINVAL), (dict(pos=None), EINVAL),
    (dict(pos=P + 2), EINVAL), (dict(table=None), EINVAL), (dict(table=P + 8), EINVAL),
    (dict(descs=[]), EINVAL), (dict(descs=[_desc(i) for i in range(5)]), EINVAL),
    (dict(descs=[_desc(heads=0)]), EINVAL), (dict(descs=[_desc(x=None)]), EINVAL), (dict(descs=[_desc(y=None)]), EINVAL),
    (dict(descs=[_desc(x=P + 2)]), EINVAL), (dict(descs=[_desc(x_tok=-512)]), EINVAL),
    (dict(descs=[_desc(y_head=64)]), EINVAL), (dict(descs=[_desc(y_tok=256)]), EINVAL),   # rows that overlap
    (dict(descs=[_desc(y_tok=0)]), EINVAL),
    (dict(descs=[_desc(y=P)]), EINVAL),                                                 # in place, another type
    (dict(descs=[_desc(y=P, y_tok=1024)], yd=0), EINVAL),                               # in place, other strides
    (dict(T=0, pos=None, table=None, descs=[_desc(x=None, y=None)]), 0)])
def test_rope_rejects(kw, want):
    assert _rope(**kw) == want


def test_rope_table_rejects():
    f = lambda freq=P, half=32, n=8, m=1.0, t=P + SLOT: K.bitlinear_rope_table(freq, half, n, m, t, None)
    assert f(half=0) == f(half=129) == f(n=-1) == f(m=math.nan) == f(freq=None) == f(t=None) == EINVAL
    assert f(freq=P + 4) == f(t=P + SLOT + 8) == f(t=P) == EINVAL
    assert f(n=(1 << 26) + 1) == EINVAL          # 2^31 entries and more
    assert f(n=0) == 0


def _kv(**kw):
    a = dict(k=P + 30 * SLOT, v=P + 40 * SLOT, ks=None, vs=None, page=16 * 5 * 128, head=16 * 128, tok=128, pages=100,
             page_size=16, heads=5, dim=128, dtype=1)
    a.update(kw)
    return K.BlKvCache(*a.values())


BAD_CACHES = [
    (dict(dtype=0), ENOTSUP), (dict(dtype=3), ENOTSUP), (dict(dim=4), EINVAL), (dict(dim=132), EINVAL),
    (dict(dim=264), EINVAL), (dict(pages=0), EINVAL), (dict(page_size=0), EINVAL), (dict(k=None), EINVAL),
    (dict(v=P + 8), EINVAL), (dict(tok=124), EINVAL), (dict(tok=64), EINVAL), (dict(head=128), EINVAL),
    (dict(page=1024), EINVAL), (dict(page=-16 * 5 * 128), EINVAL),
    (dict(dtype=2), EINVAL),                              # int8 without scales
    (dict(dtype=2, ks=P, vs=P + 2), EINVAL), (dict(dtype=2, ks=P, vs=P, dim=136, tok=144, head=2304, page=11520), EINVAL)]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_rejects(kw, want):
    assert _append(kv=_kv(**kw)) == want
    assert _attn(kv=_kv(**kw)) == want


def _append(q=None, k=None, v=None, **kw):
    arr = (K.BlRopeDesc * 3)(q or _desc(0, heads=20, x_tok=2560, y_tok=2560), k or _desc(1, heads=5, x_tok=640),
                             v or _desc(2, heads=5, x_tok=640))
    a = dict(T=4, R=128, inter=0, xd=0, qd=1, pos=P, seq=None, blocks=P, seqs=4, per=8, table=P, n=64, kv=_kv())
    a.update(kw)
    return K.bitlinear_rope_append(arr, *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(xd=2), ENOTSUP), (dict(qd=2), ENOTSUP), (dict(R=0), EINVAL), (dict(R=21), EINVAL), (dict(R=136), EINVAL),
    (dict(T=-1), EINVAL), (dict(seqs=0), EINVAL), (dict(per=0), EINVAL), (dict(blocks=None), EINVAL),
    (dict(blocks=P + 2), EINVAL), (dict(seq=P + 1), EINVAL), (dict(pos=None), EINVAL), (dict(table=P + 4), EINVAL),
    (dict(kv=None), EINVAL), (dict(k=_desc(1, heads=4)), EINVAL), (dict(v=_desc(2, heads=6)), EINVAL),
    (dict(k=_desc(1, heads=5, x=P + SLOT + 2)), EINVAL), (dict(q=_desc(0, heads=20, x_tok=2560, y_tok=640)), EINVAL)])
def test_append_rejects(kw, want):
    assert _append(**kw) == want


def _attn(plan=None, **kw):
    if plan is None:
        st, plan = K.bitlinear_paged_attn_plan(4, 20, 5, 128, 5000, 0)
        assert st == 0
    a = dict(q=P, qd=1, q_tok=2560, q_head=128, scale=0.1, kv=_kv(), blocks=P, per=8, lens=P, out=P + SLOT,
             lse=P + 2 * SLOT, ws=P + 3 * SLOT, wsb=1 << 34)
    a.update(kw)
    return K.bitlinear_paged_attn(ctypes.byref(plan), *a.values(), None)


def _changed(**kw):
    st, plan = K.bitlinear_paged_attn_plan(4, 20, 5, 128, 5000, 0)
    for k, v in kw.items():
        setattr(plan, k, v)
    return plan


@pytest.mark.parametrize("kw,want", [
    (dict(qd=2), ENOTSUP), (dict(q=None), EINVAL), (dict(q=P + 8), EINVAL), (dict(q_tok=2564), EINVAL),
    (dict(q_head=-128), EINVAL), (dict(scale=math.inf), EINVAL), (dict(per=-1), EINVAL), (dict(blocks=None), EINVAL),
    (dict(lens=None), EINVAL), (dict(out=None), EINVAL), (dict(lse=P + 2), EINVAL), (dict(ws=None), EINVAL),
    (dict(ws=P + 3 * SLOT + 128), EINVAL), (dict(wsb=255), ENOSPC), (dict(out=P + 3 * SLOT), EINVAL),
    (dict(lse=P + SLOT), EINVAL), (dict(lse=P + 3 * SLOT), EINVAL),
    (dict(out=P), EINVAL), (dict(lse=P + 8), EINVAL), (dict(out=P + 30 * SLOT), EINVAL), (dict(ws=P + 40 * SLOT), EINVAL), (dict(kv=_kv(heads=4)), EINVAL),
    (dict(kv=_kv(dim=64)), EINVAL), (dict(plan=_changed(blocks=99)), EINVAL), (dict(plan=_changed(blocks=0)), EINVAL),
    (dict(plan=_changed(B=-1)), EINVAL), (dict(plan=_changed(q_heads=21)), EINVAL)])
def test_attention_rejects(kw, want):
    assert _attn(**kw) == want


def test_attention_plan():
    f = K.bitlinear_paged_attn_plan
    for a in [(-1, 8, 8, 64, 10, 0), (1, 8, 0, 64, 10, 0), (1, 8, 3, 64, 10, 0), (1, 4, 8, 64, 10, 0),
              (1, 8, 8, 60, 10, 0), (1, 8, 8, 264, 10, 0), (1, 8, 8, 64, 0, 0), (1, 8, 8, 64, 10, -1),
              (1 << 20, 1 << 16, 1 << 16, 64, 10, 0)]:
        assert f(*a)[0] == EINVAL, a
    for B, hq, hk, D, n, w in [(1, 20, 5, 128, 262144, 0), (64, 32, 8, 128, 8192, 0), (1, 1, 1, 8, 1, 0),
                               (3, 500, 25, 64, 100000, 77), (1, 1, 1, 128, 2 ** 31 - 1, 0)]:
        st, p = f(B, hq, hk, D, n, w)
        tiles = B * hk * -(-hq // hk // 16) * (-(-(min(n, w) if w else n) // 128) + 6)
        assert st == 0 and 1 <= p.blocks <= max(1, tiles) and p.ws_bytes >= 256
        # tickets, then two partial sums per block
        assert p.ws_bytes >= 4 * B * hk + 2 * p.blocks * (128 + 4 * D * min(16, hq // hk))
    assert f(0, 8, 8, 64, 10, 0)[0] == 0


# ---- the torch wrappers ----

class Strided(FakeT):
    """A stand-in with strides, contiguous unless given otherwise."""

    def __init__(self, shape, dtype, strides=None, device=DEV):
        super().__init__(shape, dtype, device)
        want, n = [], 1
        for d in reversed(self.shape):
            want.insert(0, n)
            n *= d
        self._s = tuple(want) if strides is None else tuple(strides)
        self._contig = self._s == tuple(want)

    def stride(self, i=None):
        return self._s if i is None else self._s[i]

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def new_empty(self, shape, dtype=None):
        return Strided(shape, dtype or self.dtype, device=self.device)


F32, BF, I8, I32 = torch.float32, torch.bfloat16, torch.int8, torch.int32


def test_norm_wrappers_reject():
    x, w, r = Strided((4, 256), F32), Strided(256, F32), Strided((4, 256), BF)
    out = (Strided((4, 256), I8), Strided(4, F32), Strided((4, 256), BF), None)
    for a, kw in [((Strided((4, 256), torch.float16),), {}), ((Strided((4, 2, 128), F32),), {}),
                  ((Strided((4, 256), F32, (512, 1)),), {}), ((x, Strided(255, F32)), {}), ((x, Strided(256, BF)), {}),
                  ((x, w, Strided((3, 256), BF)), {}), ((x, w, Strided((4, 256), BF, device=torch.device("cuda:1"))), {}),
                  ((x, w, r), dict(out=(out[0], out[1], None, None))), ((x, w), dict(out=out)),
                  ((x, w, r), dict(out=(Strided((4, 255), I8),) + out[1:])),
                  ((x, w, r), dict(out=(out[0], Strided(3, F32)) + out[2:])),
                  ((x, w, r), dict(out=out[:2] + (Strided((4, 256), F32), None))),
                  ((x, w, r), dict(out=out[:3] + (Strided(3, F32),)))]:
        with pytest.raises(ValueError):
            S.norm_quant(*a, **kw)
    dn, h, rs = Strided((4, 256), F32), Strided((4, 256), BF), Strided(4, F32)
    for a, kw in [((dn, Strided((4, 128), BF), rs), {}), ((dn, h, Strided(3, F32)), {}),
                  ((dn, h, rs, Strided(8, F32)), {}), ((dn, h, rs, None, Strided((4, 256), BF)), dict(dtype=F32)),
                  ((dn, h, rs), dict(out=(Strided((4, 256), BF), None))), ((dn, h, rs), dict(dtype=torch.float16,
                                                                                             out=(dn, None))),
                  ((dn, h, rs), dict(out=(dn, Strided(255, F32)))),
                  ((Strided((8192, 3200), F32), Strided((8192, 3200), BF), Strided(8192, F32)),
                   dict(out=(Strided((8192, 3200), F32), Strided(3200, F32)), ws=Strided(64, torch.uint8)))]:
        with pytest.raises(ValueError):
            S.norm_quant_bwd(*a, **kw)


def test_rope_wrappers_reject():
    x, pos, tab = Strided((4, 3, 64), F32), Strided(4, I32), Strided((50, 32, 2), F32)
    y = Strided((4, 3, 64), F32)
    for xs, p, t, kw in [([], pos, tab, {}), ([Strided((4, 64), F32)], pos, tab, {}), ([x], Strided(3, I32), tab, {}),
                         ([x], Strided(4, torch.int64), tab, {}), ([x], pos, Strided((50, 64), F32), {}),
                         ([x], pos, Strided((50, 32, 2), torch.float64), {}),
                         ([x, Strided((4, 3, 64), BF)], pos, tab, dict(outs=[y, y])),
                         ([x, Strided((5, 3, 64), F32)], pos, tab, dict(outs=[y, y])),
                         ([x], pos, tab, dict(outs=[y, y])), ([x], pos, tab, dict(outs=[Strided((4, 2, 64), F32)])),
                         ([x], pos, tab, dict(outs=[y], dtype=BF)),
                         ([Strided((4, 3, 64), F32, (384, 128, 2))], pos, tab, dict(outs=[y]))]:
        with pytest.raises(ValueError):
            S.rope(xs, p, t, **kw)
    with pytest.raises(ValueError):
        S.rope_table(4, Strided(32, F32), out=Strided((4, 32, 2), F32))
    with pytest.raises(ValueError):
        S.rope_table(4, Strided(32, torch.float64), out=Strided((4, 31, 2), F32))
    for a in [(7,), (64, 1.0), (64, 10000.0, 0.5), (64, 10000.0, 2.0, "other")]:
        with pytest.raises(ValueError):
            S.rope_frequencies(*a)


def _cache_args(**kw):
    a = dict(q=Strided((4, 8, 64), BF), k=Strided((4, 2, 64), BF), v=Strided((4, 2, 64), BF), pos=Strided(4, I32),
             table=Strided((50, 32, 2), F32), kc=Strided((9, 2, 16, 64), BF), vc=Strided((9, 2, 16, 64), BF),
             blocks=Strided((4, 2), I32))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,opt", [
    (dict(q=Strided((4, 512), BF)), {}), (dict(k=Strided((4, 3, 64), BF)), {}), (dict(v=Strided((4, 2, 64), F32)), {}),
    (dict(pos=Strided(4, torch.int64)), {}), (dict(blocks=Strided(8, I32)), {}), (dict(blocks=Strided((4, 2), F32)), {}),
    (dict(kc=Strided((9, 2, 16, 64), F32), vc=Strided((9, 2, 16, 64), F32)), {}),
    (dict(vc=Strided((8, 2, 16, 64), BF)), {}), (dict(kc=Strided((9, 2, 16, 64), BF, (1, 2, 3, 4))), {}),
    (dict(kc=Strided((9, 2, 16, 32), BF), vc=Strided((9, 2, 16, 32), BF)), {}),
    (dict(kc=Strided((9, 2, 16, 64), I8), vc=Strided((9, 2, 16, 64), I8)), {}), ({}, dict(k_scale=Strided((9, 2, 16), F32))),
    (dict(kc=Strided((9, 2, 16, 64), I8), vc=Strided((9, 2, 16, 64), I8)),
     dict(k_scale=Strided((9, 2, 15), F32), v_scale=Strided((9, 2, 16), F32))),
    ({}, dict(seq=Strided(3, I32))), ({}, dict(dtype=F32))])
def test_append_wrapper_rejects(kw, opt):
    opt = dict(dict(out=Strided((4, 8, 64), BF)), **opt)
    with pytest.raises(ValueError):
        S.rope_append(*_cache_args(**kw).values(), **opt)


def test_attention_wrapper_rejects():
    with pytest.raises(S.BitLinearError):
        S.PagedAttn(1, 7, 2, 64, 16, 100, device="cpu")
    plan = S.PagedAttn(4, 8, 2, 64, 16, 100, device="cpu")
    plan.ws = Strided(plan.plan.ws_bytes, torch.uint8)
    ok = dict(q=Strided((4, 8, 64), BF), kc=Strided((9, 2, 16, 64), BF), vc=Strided((9, 2, 16, 64), BF),
              blocks=Strided((4, 2), I32), lens=Strided(4, I32))
    out = Strided((4, 8, 64), BF)
    for kw, opt in [(dict(q=Strided((4, 8, 32), BF)), {}), (dict(q=Strided((4, 8, 64), torch.float16)), {}),
                    (dict(q=Strided((3, 8, 64), BF)), {}), (dict(blocks=Strided((3, 2), I32)), {}),
                    (dict(blocks=Strided((4, 2), torch.int64)), {}), (dict(lens=Strided(3, I32)), {}),
                    (dict(kc=Strided((9, 2, 8, 64), BF), vc=Strided((9, 2, 8, 64), BF)), {}),
                    ({}, dict(out=Strided((4, 8, 64), F32))), ({}, dict(lse=Strided((4, 7), F32))),
                    ({}, dict(k_scale=Strided((9, 2, 16), F32)))]:
        with pytest.raises(ValueError):
            plan(*dict(ok, **kw).values(), **dict(dict(out=out), **opt))


# ---- pins of the plain implementations ----

def test_norm_gradient_formula_against_differences():
    g = np.random.default_rng(0)
    h, dn, w = g.standard_normal((3, 24)), g.standard_normal((3, 24)), 1 + 0.3 * g.standard_normal(24)
    rstd = 1 / np.sqrt((h * h).mean(-1) + 1e-3)
    dh, dw = R.norm_grad(dn, h, rstd, w)
    f = lambda a, b: (dn * R.norm_rows(a, b, 1e-3)).sum()
    e = 1e-6
    for t in range(3):
        for k in range(0, 24, 5):
            d = np.zeros((3, 24))
            d[t, k] = e
            assert abs((f(h + d, w) - f(h - d, w)) / (2 * e) - dh[t, k]) < 1e-7
    for k in range(24):
        d = np.zeros(24)
        d[k] = e
        assert abs((f(h, w + d) - f(h, w - d)) / (2 * e) - dw[k]) < 1e-7


def test_rope_reference_turns_by_the_angle():
    x = np.zeros((2, 1, 8), np.float32)
    x[:, 0, 0] = 1.0
    x[:, 0, 7] = 5.0
    f, m = S.rope_frequencies(4, 100.0)
    assert f == [1.0, 0.1] and m == 1.0
    table = R.rope_table(f, 10)
    for inter, other in ((False, 2), (True, 1)):
        y = R.rope(x, [3, 0], table, inter)
        assert abs(y[0, 0, 0] - math.cos(3)) < 1e-7 and abs(y[0, 0, other] - math.sin(3)) < 1e-7
        assert y[0, 0, 7] == 5.0 and np.array_equal(y[1], x[1])
        assert np.allclose(R.rope(y, [3, 0], table, inter, True), x, atol=1e-7)


def test_rope_frequency_scaling():
    plain, _ = S.rope_frequencies(64)
    lin, m = S.rope_frequencies(64, factor=4.0, scaling="linear")
    assert m == 1.0 and np.allclose(np.array(lin) * 4, plain)
    raised, _ = S.rope_frequencies(64, factor=4.0, scaling="base")
    assert raised[0] == plain[0] and abs(raised[-1] * 4 / plain[-1] - 1) < 1e-12
    parts, m = S.rope_frequencies(64, factor=4.0, scaling="parts", trained=2048)
    ratio = np.array(parts) / plain
    assert ratio[0] == 1.0 and abs(ratio[-1] - 0.25) < 1e-12 and np.all(np.diff(ratio) <= 1e-15)
    assert abs(m - (0.1 * math.log(4.0) + 1)) < 1e-12


def test_attention_reference_against_a_dense_softmax():
    g = np.random.default_rng(1)
    q = g.standard_normal((1, 4, 8)).astype(np.float32)
    kc, vc = g.standard_normal((3, 2, 5, 8)), g.standard_normal((3, 2, 5, 8))
    blocks = np.array([[2, 0, 1]])
    out, lse, _, _ = R.paged_attn(q, kc, vc, blocks, [12], 0.5)
    order = [(2, i) for i in range(5)] + [(0, i) for i in range(5)] + [(1, 0), (1, 1)]
    for h in range(4):
        k = np.array([kc[p, h // 2, i] for p, i in order])
        v = np.array([vc[p, h // 2, i] for p, i in order])
        e = np.exp(0.5 * k @ q[0, h].astype(np.float64))
        assert np.allclose(out[0, h], e @ v / e.sum()) and abs(lse[0, h] - np.log(e.sum())) < 1e-12
    out, lse, _, _ = R.paged_attn(q, kc, vc, np.array([[-1, 5, 3]]), [12], 0.5)
    assert not out.any() and np.all(np.isneginf(lse))
