"""ctypes binding of the operators around a model's blocks: what turns requests and token ids into the
first block's input, and the last block's output into the next token ids.

Raw calls mirror the C ABI (``include/bitlinear.h``): ``bitlinear_kv_step``, ``bitlinear_embed``,
``bitlinear_embed_bwd_workspace_bytes``, ``bitlinear_embed_bwd``, ``bitlinear_q4_bytes``,
``bitlinear_q4_pack``, ``bitlinear_q4_fwd``, ``bitlinear_sample_workspace_bytes``, ``bitlinear_sample``.
``kv_step`` / ``embed`` / ``embed_bwd`` / ``q4_pack`` / ``q4_fwd`` / ``sample`` take torch tensors, check them (the
C ABI receives bare pointers), allocate outputs that are not given and enqueue on torch's current stream.  Every step runs in HIP kernels.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

from . import bitlinear as _B
from .bitlinear import _check, _ptr
from .block import _F32, _I32, _I64, _SZ, _VP, _buf, _device, _dt, _enqueue, _rows

BL_EMBED_ACCUM = 1

_fns = None


def _lib():
    """The library, with these calls' argument types declared."""
    global _fns
    if _fns is None:
        L = _B.lib()
        L.bitlinear_kv_step.argtypes = [_VP, _VP, _I64, _VP, _I64, _I64, _VP, _I64, _VP, _VP, _I64, _VP,
                                        _VP, _VP, _VP, _VP, _VP]
        L.bitlinear_embed.argtypes = [_VP, _I32, _I64, _I64, _VP, _I64, _F32, _VP, _I32, _VP]
        L.bitlinear_embed_bwd_workspace_bytes.argtypes = [_I64, _I64, ctypes.POINTER(_SZ)]
        L.bitlinear_embed_bwd.argtypes = [_VP, _I32, _VP, _I64, _I64, _I64, _F32, _VP, _I32, _VP, _SZ, _VP]
        szp = ctypes.POINTER(_SZ)
        L.bitlinear_q4_bytes.argtypes = [_I64, _I64, _I32, szp, szp]
        L.bitlinear_q4_pack.argtypes = [_VP, _I32, _I64, _I64, _I32, _VP, _VP, _VP]
        L.bitlinear_q4_fwd.argtypes = [_VP, _VP, _I64, _I64, _VP, _VP, _I32, _I64, _VP, _VP]
        L.bitlinear_sample_workspace_bytes.argtypes = [_I64, _I64, szp]
        L.bitlinear_sample.argtypes = [_VP, _I32, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]
        for f in (L.bitlinear_kv_step, L.bitlinear_embed, L.bitlinear_embed_bwd_workspace_bytes, L.bitlinear_embed_bwd,
                  L.bitlinear_q4_bytes, L.bitlinear_q4_pack, L.bitlinear_q4_fwd, L.bitlinear_sample_workspace_bytes,
                  L.bitlinear_sample):
            f.restype = ctypes.c_int
        _fns = L
    return _fns


# ---------------------------------------------------------------------------------------------
# raw C ABI (integers and pointers)
# ---------------------------------------------------------------------------------------------

def bitlinear_kv_step(cached, fresh, B, blocks, blocks_per_seq, page_size, free_pages, free_cap, free_count,
                      free_count_out, T, seq, pos, slot, lens, starts, stream) -> int:
    return _lib().bitlinear_kv_step(cached, fresh, B, blocks, blocks_per_seq, page_size, free_pages, free_cap,
                                    free_count, free_count_out, T, seq, pos, slot, lens, starts, stream)


def bitlinear_embed(table, table_dtype, V, K, ids, T, scale, y, y_dtype, stream) -> int:
    return _lib().bitlinear_embed(table, table_dtype, V, K, ids, T, scale, y, y_dtype, stream)


def bitlinear_embed_bwd_workspace_bytes(T, K):
    """Returns (status, ws_bytes)."""
    ws = _SZ()
    st = _lib().bitlinear_embed_bwd_workspace_bytes(T, K, ctypes.byref(ws))
    return st, ws.value


def bitlinear_embed_bwd(dy, dy_dtype, ids, T, V, K, scale, dtable, flags, ws, ws_bytes, stream) -> int:
    return _lib().bitlinear_embed_bwd(dy, dy_dtype, ids, T, V, K, scale, dtable, flags, ws, ws_bytes, stream)


def bitlinear_q4_bytes(n, K, group):
    """Returns (status, code_bytes, scale_bytes)."""
    c, s = _SZ(), _SZ()
    st = _lib().bitlinear_q4_bytes(n, K, group, ctypes.byref(c), ctypes.byref(s))
    return st, c.value, s.value


def bitlinear_q4_pack(W, w_dtype, n, K, group, codes, scales, stream) -> int:
    return _lib().bitlinear_q4_pack(W, w_dtype, n, K, group, codes, scales, stream)


def bitlinear_q4_fwd(xq, x_scale, T, K, codes, scales, group, n, y, stream) -> int:
    return _lib().bitlinear_q4_fwd(xq, x_scale, T, K, codes, scales, group, n, y, stream)


def bitlinear_sample_workspace_bytes(B, V):
    """Returns (status, ws_bytes)."""
    ws = _SZ()
    st = _lib().bitlinear_sample_workspace_bytes(B, V, ctypes.byref(ws))
    return st, ws.value


def bitlinear_sample(x, x_dtype, B, V, row_stride, temperature, top_k, top_p, min_p, u, token, logprob, ws,
                     ws_bytes, stream) -> int:
    return _lib().bitlinear_sample(x, x_dtype, B, V, row_stride, temperature, top_k, top_p, min_p, u, token, logprob,
                                   ws, ws_bytes, stream)


# ---------------------------------------------------------------------------------------------
# torch convenience wrappers
# ---------------------------------------------------------------------------------------------

class KvStep(NamedTuple):
    """What ``kv_step`` returns: token rows (seq, pos int32 [T], slot int64 [T]) as ``rope_append`` takes
    them, lens (int32 [B]) as ``PagedAttn`` does, starts (int32 [B + 1]) and the free pages left."""
    seq: object
    pos: object
    slot: object
    lens: object
    starts: object
    count: object


def kv_step(cached, fresh, blocks, free, count, page_size: int, T: int, out=None) -> KvStep:
    """Pages and slots of a step's tokens, from request lengths on the GPU (all tensors int32).

    Request b has cached[b] tokens in the cache and adds fresh[b]; below 0 it has ended and its pages go
    back.  blocks [B][blocks per sequence] and free (a stack of free pages, its first count[0] entries)
    are updated in place; new pages come from the stack's top.  Requests whose pages or token rows do not
    suffice are left out (lens[b] == cached[b]).  T is the number of token rows; those no request fills
    are -1.  ``out`` may supply a ``KvStep`` (slot may be None: not wanted); its lens may be ``cached`` and
    its count ``count`` (in place, for steps that are replayed as a graph).
    """
    import torch
    i32 = torch.int32
    if len(blocks.shape) != 2:
        raise ValueError("blocks: must be [B][blocks per sequence]")
    B, per = blocks.shape
    ix = _device(blocks, "blocks")
    _buf(blocks, i32, 0, ix, "blocks")
    _buf(cached, i32, B, ix, "cached")
    _buf(fresh, i32, B, ix, "fresh")
    _buf(free, i32, 0, ix, "free")
    _buf(count, i32, 1, ix, "count")
    if T < 0:
        raise ValueError(f"T: must not be negative, got {T}")
    if out is None:
        # one allocation: slot first, for its alignment
        buf = blocks.new_empty(4 * T + 2 * B + 2)
        slot, seq, pos, lens, starts, left = buf.split_with_sizes((2 * T, T, T, B, B + 1, 1))
        out = KvStep(seq, pos, slot.view(torch.int64), lens, starts, left)
    else:
        _buf(out.seq, i32, T, ix, "seq")
        _buf(out.pos, i32, T, ix, "pos")
        if out.slot is not None:
            _buf(out.slot, torch.int64, T, ix, "slot")
        _buf(out.lens, i32, B, ix, "lens")
        _buf(out.starts, i32, B + 1, ix, "starts")
        _buf(out.count, i32, 1, ix, "count")
    _enqueue(ix, "bitlinear_kv_step", _lib().bitlinear_kv_step, cached.data_ptr(), fresh.data_ptr(), B,
             blocks.data_ptr(), per, page_size, free.data_ptr(), free.numel(), count.data_ptr(),
             out.count.data_ptr(), T, out.seq.data_ptr(), out.pos.data_ptr(), _ptr(out.slot),
             out.lens.data_ptr(), out.starts.data_ptr())
    return out


def _table(t, name: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: must be [V][K], got {tuple(shape)}")
    return shape


def embed(ids, table, scale: float = 1.0, dtype=None, out=None):
    """scale * table[ids] of int32 ids [T] and a table [V][K] (fp32 or bf16): [T][K] in ``dtype`` (that of
    the table).  An id below 0 gives a row of 0 (padding), one of V or more a row of NaN.  ``out`` may
    supply the rows."""
    import torch
    V, K = _table(table, "table")
    ix = _device(table, "table")
    td = _rows(table, table.shape, ix, "table")
    if len(ids.shape) != 1:
        raise ValueError(f"ids: must be [T], got {tuple(ids.shape)}")
    T = ids.shape[0]
    _buf(ids, torch.int32, T, ix, "ids")
    if dtype is None:
        dtype = table.dtype if out is None else out.dtype
    yd = _dt(dtype, "dtype")
    if out is None:
        out = table.new_empty((T, K), dtype=dtype)
    else:
        _rows(out, (T, K), ix, "out", dtype)
    _enqueue(ix, "bitlinear_embed", _lib().bitlinear_embed, table.data_ptr(), td, V, K, ids.data_ptr(), T,
             scale, out.data_ptr(), yd)
    return out


def embed_bwd(dy, ids, V: int, scale: float = 1.0, accumulate: bool = False, out=None, ws=None):
    """Gradient of ``embed`` for its table: fp32 [V][K] of scale * (the sum of the rows dy[t] of each id).

    dy [T][K] fp32 or bf16; ids outside [0, V) have no row.  ``accumulate`` adds to ``out``, which must
    be given then.  ``ws`` may supply a uint8 workspace, for one call at a time.  Results do not vary from run to run.
    """
    import torch
    T, K = _table(dy, "dy")
    ix = _device(dy, "dy")
    gd = _rows(dy, dy.shape, ix, "dy")
    if ids.shape != (T,):
        raise ValueError(f"ids: must be [{T}], got {tuple(ids.shape)}")
    _buf(ids, torch.int32, T, ix, "ids")
    if out is None:
        if accumulate:
            raise ValueError("out: must be given to be added to")
        out = dy.new_empty((V, K), dtype=torch.float32)
    else:
        _rows(out, (V, K), ix, "out", torch.float32)
    st, wsb = bitlinear_embed_bwd_workspace_bytes(T, K)
    _check(st, "bitlinear_embed_bwd_workspace_bytes")
    if ws is None:
        ws = dy.new_empty(wsb, dtype=torch.uint8)
    else:
        _buf(ws, torch.uint8, wsb, ix, "ws")
    _enqueue(ix, "bitlinear_embed_bwd", _lib().bitlinear_embed_bwd, dy.data_ptr(), gd, ids.data_ptr(), T, V, K,
             scale, out.data_ptr(), BL_EMBED_ACCUM if accumulate else 0, ws.data_ptr(), ws.numel())
    return out


_q4_sizes = functools.lru_cache(maxsize=64)(bitlinear_q4_bytes)


def q4_pack(W, group: int = 64, out=None):
    """W [n][K] (fp32 or bf16) in 4 bits with a bf16 scale per ``group`` (32, 64 or 128) columns of a row.

    Returns (codes uint8, scales bf16), laid out as ``q4_fwd`` takes them; ``out`` may supply them."""
    import torch
    n, K = _table(W, "W")
    ix = _device(W, "W")
    wd = _rows(W, W.shape, ix, "W")
    st, cb, sb = _q4_sizes(n, K, group)
    _check(st, "bitlinear_q4_bytes")
    if out is None:
        out = W.new_empty(cb, dtype=torch.uint8), W.new_empty(sb // 2, dtype=torch.bfloat16)
    codes, scales = out
    _buf(codes, torch.uint8, cb, ix, "codes")
    _buf(scales, torch.bfloat16, sb // 2, ix, "scales")
    _enqueue(ix, "bitlinear_q4_pack", _lib().bitlinear_q4_pack, W.data_ptr(), wd, n, K, group, codes.data_ptr(),
             scales.data_ptr())
    return codes, scales


def q4_fwd(xq, scale, K: int, codes, scales, n: int, group: int = 64, out=None):
    """y [T][n] fp32 of int8 rows xq [T][K] with their scales [T] (``norm_quant``'s or ``act_quant``'s) and
    weights from ``q4_pack``.  ``out`` may supply y."""
    import torch
    if len(xq.shape) != 2 or xq.shape[1] != K:
        raise ValueError(f"xq: must be [T][{K}], got {tuple(xq.shape)}")
    T = xq.shape[0]
    ix = _device(xq, "xq")
    _buf(xq, torch.int8, T * K, ix, "xq")
    _buf(scale, torch.float32, T, ix, "scale")
    st, cb, sb = _q4_sizes(n, K, group)
    _check(st, "bitlinear_q4_bytes")
    _buf(codes, torch.uint8, cb, ix, "codes")
    _buf(scales, torch.bfloat16, sb // 2, ix, "scales")
    if out is None:
        out = scale.new_empty((T, n))
    else:
        _rows(out, (T, n), ix, "out", torch.float32)
    _enqueue(ix, "bitlinear_q4_fwd", _lib().bitlinear_q4_fwd, xq.data_ptr(), scale.data_ptr(), T, K,
             codes.data_ptr(), scales.data_ptr(), group, n, out.data_ptr())
    return out


_sample_ws = functools.lru_cache(maxsize=64)(bitlinear_sample_workspace_bytes)


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, want_logprob: bool = False, out=None,
           ws=None):
    """A token per row of logits [B][V] (fp32 or bf16, any row stride): (int32 [B], log probabilities or None).

    u (fp64 [B], in [0, 1)) draws the tokens: the same numbers give the same tokens.  Each row has its own
    settings, tensors [B]: temperature (fp32; 0: the largest logit), top_k (int32; 0: off), top_p (fp32; 1: off), min_p
    (fp32; 0: off), applied in this order; None: 1, and off.  Logits that are -inf or NaN are masked; a row of
    them gives -1.  The log probability (fp32 [B]) is that of the token under the logits themselves.  ``out``
    may supply (tokens, log probabilities or None), ``ws`` a uint8 workspace, for one call at a time.
    """
    import torch
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError(f"logits: must be [B][V], got {tuple(shape)}")
    B, V = shape
    ix = _device(logits, "logits")
    xd = _dt(logits.dtype, "logits")
    s = logits.stride()
    if s[1] != 1 and V > 1:
        raise ValueError("logits: the last dimension must be contiguous")
    _buf(u, torch.float64, B, ix, "u")
    if temperature is not None:
        _buf(temperature, torch.float32, B, ix, "temperature")
    if top_k is not None:
        _buf(top_k, torch.int32, B, ix, "top_k")
    if top_p is not None:
        _buf(top_p, torch.float32, B, ix, "top_p")
    if min_p is not None:
        _buf(min_p, torch.float32, B, ix, "min_p")
    if out is None:
        token = u.new_empty(B, dtype=torch.int32)
        logprob = u.new_empty(B, dtype=torch.float32) if want_logprob else None
    else:
        token, logprob = out
        _buf(token, torch.int32, B, ix, "token")
        if logprob is not None:
            _buf(logprob, torch.float32, B, ix, "logprob")
    st, wsb = _sample_ws(B, V)
    _check(st, "bitlinear_sample_workspace_bytes")
    if ws is None:
        ws = u.new_empty(wsb, dtype=torch.uint8)
    else:
        _buf(ws, torch.uint8, wsb, ix, "ws")
    _enqueue(ix, "bitlinear_sample", _lib().bitlinear_sample, logits.data_ptr(), xd, B, V, s[0],
             _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p), u.data_ptr(), token.data_ptr(), _ptr(logprob),
             ws.data_ptr(), ws.numel())
    return token, logprob
