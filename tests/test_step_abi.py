"""Refusals of the operators around a model's blocks (CPU only): the C ABI rejects bad arguments before it
touches the HIP runtime (fake, never dereferenced device addresses are passed), and the torch wrappers
reject wrong tensors before anything reaches the C ABI."""
import contextlib
import math

import numpy as np
import pytest
import torch

import oracle.step_ref as R
import sparsity_amd as S
from sparsity_amd import step as K
from test_block_abi import BF, F32, I8, I32, Strided

P = 1 << 40                                # fake, 256-byte aligned; buffers 16 GiB apart
SLOT = 16 << 30
EINVAL, ENOTSUP, ENOSPC = -22, -95, -28
NAN, INF = math.nan, math.inf


def _kv(**kw):
    a = dict(cached=P, fresh=P + SLOT, B=4, blocks=P + 2 * SLOT, per=8, page=16, free=P + 3 * SLOT, cap=64,
             count=P + 4 * SLOT, left=P + 5 * SLOT, T=100, seq=P + 6 * SLOT, pos=P + 7 * SLOT, slot=P + 8 * SLOT,
             lens=P + 9 * SLOT, starts=P + 10 * SLOT)
    a.update(kw)
    return K.bitlinear_kv_step(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(B=(1 << 20) + 1), dict(T=-1), dict(T=1 << 22), dict(per=0), dict(per=1 << 31), dict(page=0),
    dict(page=1 << 31), dict(cap=-1), dict(cap=1 << 31), dict(B=1 << 20, per=1 << 20), dict(cached=None),
    dict(cached=P + 2), dict(fresh=None), dict(fresh=P + SLOT + 1), dict(blocks=None), dict(free=None),
    dict(count=None), dict(count=P + 4 * SLOT + 2), dict(left=None), dict(seq=None), dict(pos=None),
    dict(slot=P + 8 * SLOT + 4), dict(lens=None), dict(starts=None), dict(starts=P + 10 * SLOT + 2),
    dict(lens=P + 4), dict(lens=P + SLOT), dict(left=P + 9 * SLOT + 12),
    dict(left=P), dict(blocks=P + 12), dict(free=P + SLOT + 8), dict(free=P + 2 * SLOT + 4 * 8 * 4 - 4),
    dict(seq=P + 6 * SLOT, pos=P + 6 * SLOT + 396), dict(slot=P + 7 * SLOT + 392), dict(starts=P + 9 * SLOT + 12),
    dict(starts=P), dict(seq=P + 2 * SLOT), dict(pos=P + 3 * SLOT + 252), dict(slot=P + 4 * SLOT), dict(lens=P + 2 * SLOT)])
def test_kv_step_rejects(kw):
    assert _kv(**kw) == EINVAL


def _embed(**kw):
    a = dict(table=P, td=0, V=100, K=256, ids=P + SLOT, T=4, scale=1.0, y=P + 2 * SLOT, yd=1)
    a.update(kw)
    return K.bitlinear_embed(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(td=2), ENOTSUP), (dict(yd=-1), ENOTSUP), (dict(K=12), EINVAL), (dict(K=0), EINVAL), (dict(K=32776), ENOTSUP),
    (dict(T=-1), EINVAL), (dict(T=1 << 22), EINVAL), (dict(V=0), EINVAL), (dict(V=1 << 31), EINVAL),
    (dict(scale=NAN), EINVAL), (dict(scale=-INF), EINVAL), (dict(table=None), EINVAL), (dict(table=P + 8), EINVAL),
    (dict(ids=None), EINVAL), (dict(ids=P + SLOT + 2), EINVAL), (dict(y=None), EINVAL), (dict(y=P + 2 * SLOT + 4), EINVAL),
    (dict(y=P), EINVAL), (dict(y=P + 100 * 1024 - 16), EINVAL), (dict(y=P + SLOT), EINVAL),
    (dict(T=0, table=None, ids=None, y=None), 0)])
def test_embed_rejects(kw, want):
    assert _embed(**kw) == want


def _embed_bwd(**kw):
    a = dict(dy=P, dd=0, ids=P + SLOT, T=100, V=50, K=256, scale=1.0, dtable=P + 2 * SLOT, flags=0, ws=P + 3 * SLOT,
             wsb=1 << 24)
    a.update(kw)
    return K.bitlinear_embed_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dd=2), ENOTSUP), (dict(K=100), EINVAL), (dict(K=1 << 16), ENOTSUP), (dict(T=-2), EINVAL),
    (dict(T=1 << 22), EINVAL), (dict(V=0), EINVAL), (dict(V=1 << 31), EINVAL), (dict(scale=INF), EINVAL),
    (dict(flags=2), EINVAL), (dict(dy=None), EINVAL), (dict(dy=P + 2), EINVAL), (dict(ids=None), EINVAL),
    (dict(dtable=None), EINVAL), (dict(dtable=P + 2 * SLOT + 8), EINVAL), (dict(ws=None), EINVAL),
    (dict(ws=P + 3 * SLOT + 128), EINVAL), (dict(wsb=K.bitlinear_embed_bwd_workspace_bytes(100, 256)[1] - 1), ENOSPC),
    (dict(wsb=0), ENOSPC), (dict(dtable=P), EINVAL), (dict(dtable=P + SLOT), EINVAL), (dict(ws=P), EINVAL),
    (dict(ws=P + 2 * SLOT + 256), EINVAL), (dict(ws=P + SLOT), EINVAL),
    (dict(T=0, flags=1, dy=None, ids=None, dtable=None, ws=None, wsb=0), 0)])
def test_embed_grad_rejects(kw, want):
    assert _embed_bwd(**kw) == want


def test_embed_grad_workspace():
    assert K.bitlinear_embed_bwd_workspace_bytes(0, 64) == (0, 0)
    for bad in ((-1, 64), (4, 12), (1 << 22, 64)):
        assert K.bitlinear_embed_bwd_workspace_bytes(*bad)[0] == EINVAL
    assert K.bitlinear_embed_bwd_workspace_bytes(4, 1 << 16)[0] == ENOTSUP
    sizes = [K.bitlinear_embed_bwd_workspace_bytes(T, 64) for T in (1, 32, 33, 1024, 1025, 16384, 16385, (1 << 22) - 1)]
    assert all(st == 0 and n % 256 == 0 for st, n in sizes) and [n for _, n in sizes] == sorted(n for _, n in sizes)


# ---- the torch wrappers ----

def _kv_args(**kw):
    a = dict(cached=Strided(4, I32), fresh=Strided(4, I32), blocks=Strided((4, 8), I32), free=Strided(64, I32),
             count=Strided(1, I32), page=16, T=100)
    a.update(kw)
    return a


I64 = torch.int64
OUT = S.KvStep(Strided(100, I32), Strided(100, I32), Strided(100, I64), Strided(4, I32), Strided(5, I32), Strided(1, I32))
OTHER = torch.device("cuda:1")


@pytest.mark.parametrize("kw", [
    dict(blocks=Strided(32, I32)), dict(blocks=Strided((4, 8), I64)), dict(blocks=Strided((4, 8), I32, (16, 1))),
    dict(blocks=Strided((4, 8), I32, device=torch.device("cpu"))), dict(cached=Strided(3, I32)),
    dict(cached=Strided(4, I64)), dict(fresh=Strided(4, I32, device=OTHER)), dict(fresh=Strided(2, I32)),
    dict(free=Strided(64, I64)), dict(count=Strided(0, I32)), dict(count=Strided(1, I64)), dict(T=-1),
    dict(out=OUT._replace(seq=Strided(99, I32))), dict(out=OUT._replace(pos=Strided(100, I64))),
    dict(out=OUT._replace(slot=Strided(100, I32))), dict(out=OUT._replace(lens=Strided(3, I32))),
    dict(out=OUT._replace(starts=Strided(4, I32))), dict(out=OUT._replace(count=None))])
def test_kv_step_wrapper_rejects(kw):
    kw = dict(kw)
    out = kw.pop("out", OUT)
    with pytest.raises(ValueError):
        S.kv_step(*_kv_args(**kw).values(), out=out)


def test_embed_wrappers_reject():
    ids, table, y = Strided(4, I32), Strided((50, 64), F32), Strided((4, 64), BF)
    for i, t, kw in [(ids, Strided(50, F32), {}), (ids, Strided((50, 64), torch.float16), {}),
                     (ids, Strided((50, 64), F32, (128, 1)), {}), (Strided(4, I64), table, {}),
                     (Strided((4, 1), I32), table, {}), (Strided(4, I32, device=OTHER), table, {}),
                     (ids, Strided((50, 64), F32, device=torch.device("cpu")), {}),
                     (ids, table, dict(out=Strided((3, 64), BF))), (ids, table, dict(dtype=F32)),
                     (ids, table, dict(out=Strided((4, 64), torch.float16)))]:
        with pytest.raises(ValueError):
            S.embed(i, t, **dict(dict(out=y), **kw))
    dy, ws, out = Strided((4, 64), BF), Strided(1 << 20, torch.uint8), Strided((50, 64), F32)
    for d, i, kw in [(Strided(4, BF), ids, {}), (Strided((4, 64), torch.float16), ids, {}), (dy, Strided(3, I32), {}),
                     (dy, Strided(4, I64), {}), (dy, ids, dict(out=Strided((49, 64), F32))),
                     (dy, ids, dict(out=Strided((50, 64), BF))), (dy, ids, dict(out=None, accumulate=True)),
                     (dy, ids, dict(ws=Strided(64, torch.uint8))), (dy, ids, dict(ws=Strided(1 << 20, I8)))]:
        with pytest.raises(ValueError):
            S.embed_bwd(d, i, 50, **dict(dict(out=out, ws=ws), **kw))
    for k in (60, 1 << 16):
        with pytest.raises(S.BitLinearError):
            S.embed_bwd(Strided((4, k), F32), ids, 50, out=Strided((50, k), F32), ws=ws)


class Placed(Strided):
    def data_ptr(self):
        return P


def _on_devices(monkeypatch, calls_of):
    """Runs calls_of(t) with tensors of devices 1, 0 and 2 while device 0 is current: a call makes its tensors'
    device current, takes that device's stream, and leaves the current device as it was."""
    now = [0]

    @contextlib.contextmanager
    def device(index):
        was, now[0] = now[0], index
        yield
        now[0] = was

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return getattr(real, name)

            def call(*args):
                calls.append((name, now[0], args[-1]))
                return 0
            return call

    real = K._lib()
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i if now[0] == i else None,
                        raising=False)
    monkeypatch.setattr(K, "_lib", lambda: Lib())
    for index in (1, 0, 2):
        calls = []
        names = calls_of(lambda shape, dtype: Placed(shape, dtype, device=torch.device("cuda", index)))  # noqa: B023
        assert [n for n, _, _ in calls] == names
        assert all(d == index and s == 1000 + index for _, d, s in calls) and now == [0]


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    def calls(t):
        a = _kv_args(**{n: t(v.shape, v.dtype) for n, v in _kv_args().items() if isinstance(v, Strided)})
        S.kv_step(*a.values(), out=S.KvStep(*(t(v.shape, v.dtype) for v in OUT)))
        ids, table, ws = t(4, I32), t((50, 64), F32), t(1 << 20, torch.uint8)
        S.embed(ids, table, out=t((4, 64), BF))
        S.embed_bwd(t((4, 64), BF), ids, 50, out=table, ws=ws)
        return ["bitlinear_kv_step", "bitlinear_embed", "bitlinear_embed_bwd"]
    _on_devices(monkeypatch, calls)


# ---- pins of the plain implementations ----

def test_kv_reference_by_hand():
    """Two pages of three tokens a request: one ends, one grows into a new page, one begins, one waits."""
    blocks = np.array([[4, 5], [1, -1], [-1, -1], [-1, -1]], np.int32)
    free = np.array([7, 0, 0, 0], np.int32)
    seq, pos, slot, lens, starts, count = R.kv_step([5, 3, 0, 0], [-1, 1, 4, 1], blocks, free, 1, 3, 8)
    # pages 4 and 5 come back on top of 7: request 1 takes 5, request 2 takes 4 and 7, request 3 finds none
    assert free[:3].tolist() == [7, 4, 5] and count == 0
    assert blocks.tolist() == [[4, 5], [1, 5], [4, 7], [-1, -1]]
    assert lens.tolist() == [0, 4, 4, 0] and starts.tolist() == [0, 0, 1, 5, 5]
    assert seq.tolist() == [1, 2, 2, 2, 2, -1, -1, -1] and pos.tolist() == [3, 0, 1, 2, 3, -1, -1, -1]
    assert slot.tolist() == [15, 12, 13, 14, 21, -1, -1, -1]


def test_embed_reference_by_differences():
    g = np.random.default_rng(2)
    table, c = g.standard_normal((5, 8)), g.standard_normal((7, 8))
    ids = np.array([0, 3, 3, -1, 4, 3, 9])
    d, _, n = R.embed_grad(c, ids, 5, 2.0)
    assert n.tolist() == [1, 0, 0, 3, 1]
    f = lambda t: (np.nan_to_num(R.embed(ids, t, 2.0).astype(np.float64)) * c).sum()  # noqa: E731
    for v in range(5):
        e = np.zeros((5, 8))
        e[v, 2] = 0.5
        assert abs((f(table + e) - f(table - e)) - d[v, 2]) < 1e-5


# ---- weights in 4 bits ----

@pytest.mark.parametrize("n,cols,group,want", [
    (16, 128, 64, 0), (1, 32, 32, 0), (0, 128, 64, EINVAL), (-1, 128, 64, EINVAL), ((1 << 27) + 1, 128, 64, EINVAL),
    (16, 0, 64, EINVAL), (16, 96, 64, EINVAL), (16, 64, 128, EINVAL), (16, 1 << 17, 128, EINVAL), (16, 128, 16, ENOTSUP),
    (16, 128, 0, ENOTSUP), (16, 128, 256, ENOTSUP), (1 << 27, 128, 32, 0), (1 << 27, 256, 64, EINVAL),
    (1 << 22, 1 << 16, 128, EINVAL)])
def test_q4_sizes(n, cols, group, want):
    st, codes, scales = K.bitlinear_q4_bytes(n, cols, group)
    assert st == want
    if not st:
        blocks = -(-n // 16) * -(-cols // 128)
        assert codes == 1024 * blocks and scales == blocks * 16 * (128 // group) * 2


def _q4_pack(**kw):
    a = dict(W=P, wd=0, n=100, K=256, group=64, codes=P + SLOT, scales=P + 2 * SLOT)
    a.update(kw)
    return K.bitlinear_q4_pack(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(wd=2), ENOTSUP), (dict(group=48), ENOTSUP), (dict(n=0), EINVAL), (dict(K=200), EINVAL), (dict(W=None), EINVAL),
    (dict(W=P + 8), EINVAL), (dict(codes=None), EINVAL), (dict(codes=P + SLOT + 4), EINVAL), (dict(scales=None), EINVAL),
    (dict(scales=P + 2 * SLOT + 2), EINVAL), (dict(codes=P + 16), EINVAL), (dict(scales=P + 100 * 1024 - 16), EINVAL),
    (dict(scales=P + SLOT + 14 * 1024 - 16), EINVAL)])
def test_q4_pack_rejects(kw, want):
    assert _q4_pack(**kw) == want


def _q4_fwd(**kw):
    a = dict(xq=P, xs=P + SLOT, T=4, K=256, codes=P + 2 * SLOT, scales=P + 3 * SLOT, group=64, n=100, y=P + 4 * SLOT)
    a.update(kw)
    return K.bitlinear_q4_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(group=1), ENOTSUP), (dict(n=0), EINVAL), (dict(K=0), EINVAL), (dict(K=160), EINVAL), (dict(T=-1), EINVAL),
    (dict(T=1 << 22), EINVAL), (dict(T=1 << 20, n=1 << 20), EINVAL), (dict(T=1 << 14, n=1 << 20), EINVAL), (dict(xq=None), EINVAL), (dict(xq=P + 8), EINVAL),
    (dict(xs=None), EINVAL), (dict(xs=P + SLOT + 2), EINVAL), (dict(codes=None), EINVAL), (dict(codes=P + 2 * SLOT + 8), EINVAL),
    (dict(scales=P + 3 * SLOT + 8), EINVAL), (dict(scales=None), EINVAL), (dict(y=None), EINVAL), (dict(y=P + 4 * SLOT + 8), EINVAL),
    (dict(y=P), EINVAL), (dict(y=P + SLOT), EINVAL), (dict(y=P + 2 * SLOT + 14 * 1024 - 16), EINVAL), (dict(y=P + 3 * SLOT), EINVAL),
    (dict(T=0, xq=None, xs=None, codes=None, scales=None, y=None), 0)])
def test_q4_fwd_rejects(kw, want):
    assert _q4_fwd(**kw) == want


def test_q4_wrappers_reject():
    W, U8 = Strided((100, 256), F32), torch.uint8
    codes, scales = Strided(14 * 1024, U8), Strided(14 * 32, BF)
    for w, kw in [(Strided(256, F32), {}), (Strided((100, 256), torch.float16), {}), (Strided((100, 256), F32, (512, 1)), {}),
                  (W, dict(out=(Strided(14 * 1024 - 1, U8), scales))), (W, dict(out=(Strided(14 * 1024, I8), scales))),
                  (W, dict(out=(codes, Strided(14 * 32 - 1, BF)))), (W, dict(out=(codes, Strided(14 * 32, F32))))]:
        with pytest.raises(ValueError):
            S.q4_pack(w, **dict(dict(out=(codes, scales)), **kw))
    for k, group in ((200, 64), (256, 16)):
        with pytest.raises(S.BitLinearError):
            S.q4_pack(Strided((100, k), F32), group, out=(codes, scales))
    ok = dict(xq=Strided((4, 256), I8), scale=Strided(4, F32), K=256, codes=codes, scales=scales, n=100)
    y = Strided((4, 100), F32)
    for kw in [dict(xq=Strided(256, I8)), dict(xq=Strided((4, 128), I8)), dict(xq=Strided((4, 256), U8)), dict(scale=Strided(3, F32)),
               dict(scale=Strided(4, BF)), dict(codes=Strided(1024, U8)), dict(scales=Strided(14 * 16, BF)), dict(n=113),
               dict(scales=Strided(14 * 32, BF, device=OTHER)), dict(out=Strided((4, 99), F32)), dict(out=Strided((4, 100), BF))]:
        with pytest.raises(ValueError):
            S.q4_fwd(**dict(ok, **dict(dict(out=y), **kw)))
    with pytest.raises(S.BitLinearError):
        S.q4_fwd(**dict(ok, out=y, group=33))


def test_q4_calls_run_on_the_device_of_their_tensors(monkeypatch):
    def calls(t):
        codes, scales = t(14 * 1024, torch.uint8), t(14 * 32, BF)
        S.q4_pack(t((100, 256), F32), out=(codes, scales))
        S.q4_fwd(t((4, 256), I8), t(4, F32), 256, codes, scales, 100, out=t((4, 100), F32))
        return ["bitlinear_q4_pack", "bitlinear_q4_fwd"]
    _on_devices(monkeypatch, calls)


def test_q4_reference_layout_by_hand():
    """One element of each kind in its place."""
    q, s = np.zeros((17, 256), np.int8), np.zeros((17, 4), np.float32)
    q[3, 70], q[16, 128 + 5], s[3, 1], s[16, 2] = -3, 6, 1.0, 2.0
    codes, scales = R.q4_pack(q, s, 64)
    # row 3, block 0, column 70 = 64 + 6: step 1, h 0, dword 2, byte 2 high nibble; row 16: tile 1, block 1, column 5
    assert codes[3 * 16 + 2 * 4 + 2] == 13 << 4 and codes[(3 * 64) * 16 + 1] == 6 << 4 and np.count_nonzero(codes) == 2
    assert scales[(0 * 4 + 0) * 8 + 4 + 3] == 0x3F80 and scales[(3 * 4 + 0) * 8 + 0] == 0x4000
    q, s = R.q4_quantize(np.array([[7, -7, 3.5, 0.5, 1.5, 0.2] + [0] * 26], np.float32), 32)
    assert s[0, 0] == 1.0 and q[0, :6].tolist() == [7, -7, 4, 0, 2, 0]


# ---- sampling ----

@pytest.mark.parametrize("B,V,want", [(1, 1, 0), (65535, 1000, 0), (0, 10, 0), (-1, 10, EINVAL), (65536, 10, EINVAL),
                                      (1, 0, EINVAL), (1, -5, EINVAL), (1, 1 << 31, EINVAL),
                                      (1, (1 << 24) - 1, 0), (1, 1 << 24, EINVAL)])    # sums of 2^24 * 2^40 overflow
def test_sample_workspace(B, V, want):
    st, n = K.bitlinear_sample_workspace_bytes(B, V)
    assert st == want and (st or n % 256 == 0 and (n > 0) == (B > 0))


def _sample(**kw):
    a = dict(x=P, xd=0, B=4, V=1000, stride=1000, temp=P + SLOT, k=P + 2 * SLOT, p=P + 3 * SLOT, m=P + 4 * SLOT,
             u=P + 5 * SLOT, token=P + 6 * SLOT, logprob=P + 7 * SLOT, ws=P + 8 * SLOT, wsb=1 << 20)
    a.update(kw)
    return K.bitlinear_sample(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(xd=2), ENOTSUP), (dict(B=-1), EINVAL), (dict(B=65536), EINVAL), (dict(V=0), EINVAL), (dict(stride=999), EINVAL),
    (dict(stride=0), EINVAL), (dict(stride=(1 << 40) + 1), EINVAL), (dict(x=None), EINVAL), (dict(x=P + 2), EINVAL),
    (dict(xd=1, x=P + 1), EINVAL), (dict(temp=P + SLOT + 1), EINVAL), (dict(k=P + 2 * SLOT + 2), EINVAL),
    (dict(p=P + 3 * SLOT + 1), EINVAL), (dict(m=P + 4 * SLOT + 2), EINVAL), (dict(u=None), EINVAL),
    (dict(u=P + 5 * SLOT + 4), EINVAL), (dict(token=None), EINVAL), (dict(token=P + 6 * SLOT + 2), EINVAL),
    (dict(logprob=P + 7 * SLOT + 2), EINVAL), (dict(ws=None), EINVAL), (dict(ws=P + 8 * SLOT + 128), EINVAL),
    (dict(wsb=0), ENOSPC), (dict(wsb=K.bitlinear_sample_workspace_bytes(4, 1000)[1] - 1), ENOSPC), (dict(token=P), EINVAL),
    (dict(token=P + 15996), EINVAL), (dict(token=P + SLOT), EINVAL), (dict(logprob=P + 2 * SLOT), EINVAL),
    (dict(token=P + 5 * SLOT + 28), EINVAL), (dict(logprob=P + 6 * SLOT + 8), EINVAL), (dict(ws=P + 256), EINVAL),
    (dict(ws=P + 3 * SLOT), EINVAL), (dict(ws=P + 7 * SLOT), EINVAL), (dict(token=P + 4 * SLOT), EINVAL),
    (dict(B=0, x=None, u=None, token=None, ws=None, wsb=0), 0)])
def test_sample_rejects(kw, want):
    assert _sample(**kw) == want


def test_sample_wrapper_rejects():
    U8, F64 = torch.uint8, torch.float64
    ok = dict(logits=Strided((4, 1000), F32), u=Strided(4, F64), out=(Strided(4, I32), Strided(4, F32)), ws=Strided(1 << 20, U8))
    for kw in [dict(logits=Strided(1000, F32)), dict(logits=Strided((4, 1000), torch.float16)),
               dict(logits=Strided((4, 1000), F32, (1, 4))), dict(logits=Strided((4, 1000), F32, device=torch.device("cpu"))),
               dict(u=Strided(4, F32)), dict(u=Strided(3, F64)), dict(u=Strided(4, F64, device=OTHER)),
               dict(temperature=Strided(3, F32)), dict(temperature=Strided(4, F64)), dict(top_k=Strided(4, I64)),
               dict(top_k=Strided(1, I32)), dict(top_p=Strided(4, BF)), dict(min_p=Strided(4, I32)), dict(min_p=Strided(2, F32)),
               dict(out=(Strided(4, I64), None)), dict(out=(Strided(3, I32), None)), dict(out=(Strided(4, I32), Strided(4, BF))),
               dict(ws=Strided(64, U8)), dict(ws=Strided(1 << 20, I8))]:
        with pytest.raises(ValueError):
            S.sample(**dict(ok, **kw))
    with pytest.raises(S.BitLinearError):
        S.sample(Strided((4, 0), F32), ok["u"])


def test_sample_calls_run_on_the_device_of_their_tensors(monkeypatch):
    def calls(t):
        S.sample(t((4, 1000), F32), t(4, torch.float64), t(4, F32), out=(t(4, I32), None), ws=t(1 << 20, torch.uint8))
        return ["bitlinear_sample"]
    _on_devices(monkeypatch, calls)


def test_sample_reference_by_hand():
    """Probabilities 1/2, 1/4, 1/8, 1/8 (two equal logits)."""
    x = np.log([0.125, 0.5, 0.25, 0.125]) + 3
    x[0] = x[3]
    draw = lambda u, **kw: R.sample_row(x, u, **kw)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.49, 0.51, 0.74, 0.76, 0.87, 0.88, 0.999)] == [1, 1, 2, 2, 0, 0, 3, 3]
    assert [draw(u, k=2) for u in (0.6, 0.7, 0.999)] == [1, 2, 2]
    assert [draw(0.999, p=p) for p in (0.4, 0.6, 0.8, 0.9, 1.0)] == [1, 2, 0, 3, 3]
    assert [draw(0.999, min_p=m) for m in (0.9, 0.45, 0.2, 0.0)] == [1, 2, 3, 3]
    assert draw(0.999, k=3, p=0.7) == 2            # 0.7 of the 7/8 that top-k leaves: 0.6125 of 0.75
    assert draw(0.999, temperature=0.0) == 1
    assert abs(R.sample_row(x, 0.6)[1] - np.log(0.25)) < 1e-12
    assert R.sample_row([-np.inf, np.nan], 0.5)[:2] == (-1, -np.inf)


def test_model_example_rejects_pages_that_its_caches_lack():
    """Before it asks for a GPU: the stack would hand out pages in which no key is kept."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import model as E
    for kw in (dict(pages=37), dict(pages=31, page=5, max_len=25), dict(pages=-1)):
        with pytest.raises(ValueError, match="pages"):
            E.Model(6, **dict(dict(layers=1, vocab=100, hidden=256, heads=4, kv_heads=2, D=64, ffn=320, page=4,
                                   max_len=24), **kw))
