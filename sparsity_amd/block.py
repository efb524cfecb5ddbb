"""ctypes binding of the operators between a decoder block's projections.

Raw calls mirror the C ABI (``include/bitlinear.h``): ``bitlinear_norm_quant``,
``bitlinear_norm_quant_bwd_workspace_bytes``, ``bitlinear_norm_quant_bwd``,
``bitlinear_rope_table``, ``bitlinear_rope``, ``bitlinear_rope_append``,
``bitlinear_paged_attn_plan``, ``bitlinear_paged_attn``.  ``norm_quant`` / ``norm_quant_bwd`` /
``rope_table`` / ``rope`` / ``rope_append`` / ``PagedAttn`` take torch tensors, check them (the C ABI
receives bare pointers), allocate outputs that are not given and enqueue on torch's current stream.
Every step runs in HIP kernels.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import bitlinear as _B
from .bitlinear import BL_DTYPE_BF16, BL_DTYPE_F32, _check, _ptr

BL_DTYPE_I8 = 2
_I64, _I32, _VP, _SZ, _F64, _F32 = (ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                    ctypes.c_double, ctypes.c_float)


class BlRopeDesc(ctypes.Structure):
    """bl_rope_desc: one tensor of heads."""
    _fields_ = [("x", _VP), ("y", _VP), ("x_tok", _I64), ("x_head", _I64), ("y_tok", _I64),
                ("y_head", _I64), ("heads", _I64)]


class BlKvCache(ctypes.Structure):
    """bl_kv_cache: a paged key-value cache."""
    _fields_ = [("k", _VP), ("v", _VP), ("k_scale", _VP), ("v_scale", _VP), ("page_stride", _I64),
                ("head_stride", _I64), ("tok_stride", _I64), ("pages", _I64),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class BlAttnPlan(ctypes.Structure):
    """bl_attn_plan: the split of a decode attention and its workspace."""
    _fields_ = [("B", _I64), ("max_len", _I64), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("window", ctypes.c_int32), ("blocks", ctypes.c_int32), ("q_rows", ctypes.c_int32),
                ("ws_bytes", _SZ)]


# The same records as bytes, which the calls below pack in one go.
_ROPE = struct.Struct("QQ5q")
_ROPE3 = struct.Struct("QQ5qQQ5qQQ5q")
_KV = struct.Struct("4Q4q4i")

_fns = None


def _lib():
    """The library, with these calls' argument types declared."""
    global _fns
    if _fns is None:
        L = _B.lib()
        rd = kv = _VP                       # ctypes arrays, pointers or packed bytes
        pl = ctypes.POINTER(BlAttnPlan)
        L.bitlinear_norm_quant.argtypes = [_VP, _I32, _VP, _I32, _VP, _F64, _I64, _I64, _I32, _VP,
                                           _VP, _VP, _VP, _VP]
        L.bitlinear_norm_quant_bwd_workspace_bytes.argtypes = [_I64, _I64, ctypes.POINTER(_SZ)]
        L.bitlinear_norm_quant_bwd.argtypes = [_VP, _I32, _VP, _I32, _VP, _VP, _VP, _VP, _I32, _VP,
                                               _I64, _I64, _VP, _SZ, _VP]
        L.bitlinear_rope_table.argtypes = [_VP, _I64, _I64, _F64, _VP, _VP]
        L.bitlinear_rope.argtypes = [rd, _I64, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _VP, _VP,
                                     _I64, _VP]
        L.bitlinear_rope_append.argtypes = [rd, _I64, _I64, _I32, _I32, _I32, _VP, _VP, _VP, _I64,
                                            _I64, _VP, _I64, kv, _VP]
        L.bitlinear_paged_attn_plan.argtypes = [_I64, _I64, _I64, _I64, _I64, _I64, pl]
        L.bitlinear_paged_attn.argtypes = [pl, _VP, _I32, _I64, _I64, _F32, kv, _VP, _I64, _VP,
                                           _VP, _VP, _VP, _SZ, _VP]
        for f in (L.bitlinear_norm_quant, L.bitlinear_norm_quant_bwd_workspace_bytes,
                  L.bitlinear_norm_quant_bwd, L.bitlinear_rope_table, L.bitlinear_rope,
                  L.bitlinear_rope_append, L.bitlinear_paged_attn_plan, L.bitlinear_paged_attn):
            f.restype = ctypes.c_int
        _fns = L
    return _fns


# ---------------------------------------------------------------------------------------------
# raw C ABI (integers, pointers and descriptors)
# ---------------------------------------------------------------------------------------------

def bitlinear_norm_quant(x, x_dtype, res, res_dtype, w, eps, T, K, lift_M, h, xq, x_scale, rstd,
                         stream) -> int:
    return _lib().bitlinear_norm_quant(x, x_dtype, res, res_dtype, w, eps, T, K, lift_M, h, xq,
                                       x_scale, rstd, stream)


def bitlinear_norm_quant_bwd_workspace_bytes(T, K):
    """Returns (status, ws_bytes)."""
    ws = _SZ()
    st = _lib().bitlinear_norm_quant_bwd_workspace_bytes(T, K, ctypes.byref(ws))
    return st, ws.value


def bitlinear_norm_quant_bwd(dn, dn_dtype, h, h_dtype, rstd, w, dres, dh, grad_dtype, dw, T, K, ws,
                             ws_bytes, stream) -> int:
    return _lib().bitlinear_norm_quant_bwd(dn, dn_dtype, h, h_dtype, rstd, w, dres, dh, grad_dtype,
                                           dw, T, K, ws, ws_bytes, stream)


def bitlinear_rope_table(freq, half, positions, mscale, table, stream) -> int:
    return _lib().bitlinear_rope_table(freq, half, positions, mscale, table, stream)


def bitlinear_rope(descs, T, D, R, interleaved, inverse, x_dtype, y_dtype, pos, table, positions,
                   stream) -> int:
    """descs: a ctypes array of BlRopeDesc."""
    return _lib().bitlinear_rope(descs, len(descs), T, D, R, interleaved, inverse, x_dtype, y_dtype,
                                 pos, table, positions, stream)


def bitlinear_rope_append(qkv, T, R, interleaved, x_dtype, q_dtype, pos, seq, blocks, seqs,
                          blocks_per_seq, table, positions, kv, stream) -> int:
    """qkv: a ctypes array of three BlRopeDesc; kv: a BlKvCache."""
    return _lib().bitlinear_rope_append(qkv, T, R, interleaved, x_dtype, q_dtype, pos, seq, blocks,
                                        seqs, blocks_per_seq, table, positions,
                                        None if kv is None else ctypes.byref(kv), stream)


def bitlinear_paged_attn_plan(B, q_heads, kv_heads, head_dim, max_len, window):
    """Returns (status, BlAttnPlan)."""
    plan = BlAttnPlan()
    st = _lib().bitlinear_paged_attn_plan(B, q_heads, kv_heads, head_dim, max_len, window,
                                          ctypes.byref(plan))
    return st, plan


def bitlinear_paged_attn(plan, q, q_dtype, q_tok, q_head, scale, kv, blocks, blocks_per_seq, lens,
                         out, lse, ws, ws_bytes, stream) -> int:
    return _lib().bitlinear_paged_attn(plan, q, q_dtype, q_tok, q_head, scale,
                                       None if kv is None else ctypes.byref(kv), blocks,
                                       blocks_per_seq, lens, out, lse, ws, ws_bytes, stream)


# ---------------------------------------------------------------------------------------------
# torch convenience wrappers
#
# A decode step makes a few of these calls per layer with microseconds of GPU work each, so the
# checks read each tensor property once and name a fault only after one was found.
# ---------------------------------------------------------------------------------------------

def _enqueue(index: int, name: str, fn, *args) -> None:
    """fn(*args, stream) on torch's current stream of device `index`, which is made current for the call: the
    handle of a default stream stands for that of whichever device is."""
    import torch
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    _check(status, name)


def _dt(dtype, name: str) -> int:
    import torch
    if dtype is torch.float32:
        return BL_DTYPE_F32
    if dtype is torch.bfloat16:
        return BL_DTYPE_BF16
    raise ValueError(f"{name}: dtype must be float32 or bfloat16, got {dtype}")


def _buf(t, dtype, numel: int, index: int, name: str) -> None:
    """A contiguous tensor of a dtype with at least numel elements on CUDA device `index`."""
    if t is None:
        raise ValueError(f"{name}: buffer missing")
    if t.dtype is not dtype or t.get_device() != index or t.numel() < numel or not t.is_contiguous():
        raise ValueError(f"{name}: must be a contiguous {dtype} tensor of at least {numel} elements on "
                         f"cuda:{index}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, shape, index: int, name: str, dtype=None) -> int:
    """A contiguous tensor of exactly this shape; returns its dtype code."""
    if t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous {tuple(shape)} on cuda:{index}, got "
                         f"{tuple(t.shape)} on {t.device}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: dtype must be {dtype}, got {t.dtype}")
    return _dt(t.dtype, name)


def _device(t, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name}: must be a CUDA tensor, got {t.device}")
    return index


def norm_quant(x, weight=None, residual=None, eps: float = 1e-6, lift_M: int = 0,
               want_rstd: bool = False, out=None):
    """Residual addition, RMS norm and per-token int8 quantization of x[T][K] (fp32 or bf16).

    h = x + residual in residual's dtype; the normed rows h * rstd * weight (fp32 weight[K]) are
    quantized as ``act_quant(..., lift_M)`` would.  Returns (xq int8 [T][K_eff], scale fp32 [T], h,
    rstd); h is x itself without a residual, rstd (fp32 [T], for ``norm_quant_bwd``) is None unless
    wanted.  ``out`` may supply (xq, scale, h, rstd); its h may be ``residual`` (in place), and is
    None without a residual.
    """
    import torch
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x: must be [T][K], got {tuple(shape)}")
    T, K = shape
    ix = _device(x, "x")
    xd = _rows(x, shape, ix, "x")
    rd, h = 0, None
    if residual is not None:
        rd = _rows(residual, shape, ix, "residual")
    if weight is not None:
        _buf(weight, torch.float32, K, ix, "weight")
    ke = K // lift_M * (2 * lift_M - 4) if lift_M else K
    if out is None:
        xq = x.new_empty((T, ke), dtype=torch.int8) if lift_M else torch.empty_like(x, dtype=torch.int8)
        scale = x.new_empty(T, dtype=torch.float32)
        if residual is not None:
            h = torch.empty_like(residual)
        rstd = torch.empty_like(scale) if want_rstd else None
    else:
        xq, scale, h, rstd = out
        _buf(xq, torch.int8, T * ke, ix, "xq")
        _buf(scale, torch.float32, T, ix, "scale")
        if (h is None) != (residual is None):
            raise ValueError("h: given exactly with a residual")
        if h is not None:
            _rows(h, shape, ix, "h", residual.dtype)
        if rstd is not None:
            _buf(rstd, torch.float32, T, ix, "rstd")
    _enqueue(ix, "bitlinear_norm_quant", _lib().bitlinear_norm_quant, x.data_ptr(), xd,
             _ptr(residual), rd, _ptr(weight), eps, T, K, lift_M, _ptr(h), xq.data_ptr(),
             scale.data_ptr(), _ptr(rstd))
    return xq, scale, x if h is None else h, rstd


def norm_quant_bwd(dn, h, rstd, weight=None, dres=None, dtype=None, want_dw: bool = True, out=None,
                   ws=None):
    """Gradient of ``norm_quant``, straight through the quantizer: (dh, dw).

    dn[T][K] (fp32 or bf16) is the gradient of the normed rows (``bwd``'s dx), h and rstd the
    forward's; dres[T][K], if given, is the gradient that reaches h along the residual stream and is
    added.  dh is the gradient of x and of the residual, in ``dtype`` (that of dres, else dn's); dw
    fp32 [K] that of the weight.  ``out`` may supply (dh, dw); dh may be dres.  ``ws`` may supply
    a uint8 workspace.
    """
    import torch
    shape = dn.shape
    if len(shape) != 2:
        raise ValueError(f"dn: must be [T][K], got {tuple(shape)}")
    T, K = shape
    ix = _device(dn, "dn")
    gd = _rows(dn, shape, ix, "dn")
    hd = _rows(h, shape, ix, "h")
    _buf(rstd, torch.float32, T, ix, "rstd")
    if weight is not None:
        _buf(weight, torch.float32, K, ix, "weight")
    if dtype is None:
        dtype = dn.dtype if dres is None else dres.dtype
    od = _dt(dtype, "dtype")
    if dres is not None:
        _rows(dres, shape, ix, "dres", dtype)
    if out is None:
        dh = torch.empty_like(dn, dtype=dtype)
        dw = dn.new_empty(K, dtype=torch.float32) if want_dw else None
    else:
        dh, dw = out
        _rows(dh, shape, ix, "dh", dtype)
        if dw is not None:
            _buf(dw, torch.float32, K, ix, "dw")
    wsb = 0
    if dw is not None:
        st, wsb = bitlinear_norm_quant_bwd_workspace_bytes(T, K)
        _check(st, "bitlinear_norm_quant_bwd_workspace_bytes")
    if wsb == 0:
        ws = None
    elif ws is None:
        ws = dn.new_empty(wsb, dtype=torch.uint8)
    else:
        _buf(ws, torch.uint8, wsb, ix, "ws")
        wsb = ws.numel()
    _enqueue(ix, "bitlinear_norm_quant_bwd", _lib().bitlinear_norm_quant_bwd, dn.data_ptr(), gd,
             h.data_ptr(), hd, rstd.data_ptr(), _ptr(weight), _ptr(dres), dh.data_ptr(), od, _ptr(dw),
             T, K, _ptr(ws), wsb)
    return dh, dw


def rope_frequencies(rot: int, base: float = 10000.0, factor: float = 1.0, scaling: str = "none",
                     trained: int = 4096, fast: float = 32.0, slow: float = 1.0):
    """The angle per position of each of the rot / 2 pairs, and the scale of cos and sin.

    scaling, for contexts ``factor`` times the ``trained`` length:
      "none"    base^(-2i / rot)
      "linear"  every frequency divided by factor (positions interpolated)
      "base"    the base raised so that the slowest pair is divided by factor, the fastest kept
      "parts"   pairs that turn more than ``fast`` times over the trained length are kept, those
                that turn fewer than ``slow`` times are divided by factor, a ramp between; cos and
                sin are scaled by 0.1 log(factor) + 1
    Returns (list of floats, float).
    """
    if rot < 2 or rot % 2 or factor < 1.0 or base <= 1.0:
        raise ValueError("rot must be even and at least 2, factor at least 1, base above 1")
    half = rot // 2
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    freq = [base ** (-2.0 * i / rot) for i in range(half)]
    if scaling in ("none", "base"):
        return freq, 1.0
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling != "parts":
        raise ValueError(f"scaling: unknown {scaling!r}")
    out = []
    for f in freq:
        turns = trained * f / (2.0 * math.pi)
        keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
        out.append(f * keep + f / factor * (1.0 - keep))
    return out, 0.1 * math.log(factor) + 1.0


def rope_table(positions: int, freq, mscale: float = 1.0, device="cuda", out=None):
    """fp32 [positions][len(freq)][2]: cos and sin of position * freq[i] times mscale, computed in
    fp64 and rounded once.  ``freq`` is a sequence of floats or an fp64 CUDA tensor
    (``rope_frequencies`` gives them)."""
    import torch
    if isinstance(freq, (list, tuple)):
        freq = torch.tensor(freq, dtype=torch.float64, device=device)
    ix = _device(freq, "freq")
    _buf(freq, torch.float64, 1, ix, "freq")
    half = freq.numel()
    if out is None:
        out = freq.new_empty((positions, half, 2), dtype=torch.float32)
    _buf(out, torch.float32, positions * half * 2, ix, "out")
    _enqueue(ix, "bitlinear_rope_table", _lib().bitlinear_rope_table, freq.data_ptr(), half,
             positions, mscale, out.data_ptr())
    return out


def _heads(t, T: int, D: int, index: int, name: str, dtype):
    """A [T][heads][D] tensor (any strides but the last): (token stride, head stride, heads)."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != D or t.get_device() != index:
        raise ValueError(f"{name}: must be [{T}][heads][{D}] on cuda:{index}, got {tuple(shape)} on "
                         f"{t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype must be {dtype}, got {t.dtype}")
    s = t.stride()
    if s[2] != 1 and D > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return s[0], s[1], shape[1]


def _like(t, dtype):
    """A new contiguous tensor of t's shape."""
    import torch
    return torch.empty_like(t, dtype=dtype) if t.is_contiguous() else t.new_empty(t.shape, dtype=dtype)


def _table(table, index: int):
    import torch
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2:
        raise ValueError(f"table: must be [positions][pairs][2], got {tuple(shape)}")
    _buf(table, torch.float32, 0, index, "table")
    return shape[0], 2 * shape[1]


def rope(xs, pos, table, interleaved: bool = False, inverse: bool = False, dtype=None, outs=None):
    """Rotary positions on up to four tensors [T][heads][D] (one dtype, any token and head strides)
    in one launch; the first 2 * table.shape[1] elements of each head are rotated.

    pos: int32 [T]; table: ``rope_table``'s.  ``inverse`` turns back, which is the gradient.
    Returns a list of tensors in ``dtype`` (that of xs); ``outs`` may supply them, and may be xs
    itself (in place).
    """
    import torch
    if not xs or len(xs[0].shape) != 3:
        raise ValueError("xs: must be tensors [T][heads][D]")
    T, _, D = xs[0].shape
    xdt = xs[0].dtype
    ix = _device(xs[0], "xs")
    positions, R = _table(table, ix)
    _buf(pos, torch.int32, T, ix, "pos")
    if dtype is None:
        dtype = xdt if outs is None else outs[0].dtype
    xd, yd = _dt(xdt, "xs"), _dt(dtype, "dtype")
    if outs is not None and len(outs) != len(xs):
        raise ValueError("outs: one per tensor")
    strides = []
    for i, x in enumerate(xs):
        xt, xh, n = _heads(x, T, D, ix, "xs", xdt)
        if outs is None:
            strides.append((xt, xh, n * D, D, n))
        else:
            yt, yh, m = _heads(outs[i], T, D, ix, "outs", dtype)
            if m != n:
                raise ValueError("outs: heads differ from xs")
            strides.append((xt, xh, yt, yh, n))
    if outs is None:
        outs = [_like(x, dtype) for x in xs]
    arr = b"".join([_ROPE.pack(x.data_ptr(), y.data_ptr(), *s)
                    for x, y, s in zip(xs, outs, strides)])
    _enqueue(ix, "bitlinear_rope", _lib().bitlinear_rope, arr, len(xs), T, D, R, interleaved, inverse,
             xd, yd, pos.data_ptr(), table.data_ptr(), positions)
    return outs


def _cache_check(k, v, k_scale, v_scale, index: int):
    """Checks of a cache's tensors [pages][heads][page_size][D] (any strides but the last, the same
    for both) and scales [pages][heads][page_size]; returns the fields of a BlKvCache behind its
    pointers."""
    import torch
    shape, s, dtype = k.shape, k.stride(), k.dtype
    if (len(shape) != 4 or shape != v.shape or dtype is not v.dtype or
            s != v.stride() and any(n > 1 and i != j for n, i, j in zip(shape, s, v.stride()))):
        raise ValueError("k_cache, v_cache: must be [pages][heads][page_size][D] with the same "
                         "shape, strides and dtype")
    if k.get_device() != index or v.get_device() != index:
        raise ValueError(f"k_cache, v_cache: must be CUDA tensors on cuda:{index}")
    pages, heads, ps, D = shape
    if s[3] != 1 and D > 1:
        raise ValueError("k_cache: the last dimension must be contiguous")
    if dtype is torch.int8:
        _buf(k_scale, torch.float32, pages * heads * ps, index, "k_scale")
        _buf(v_scale, torch.float32, pages * heads * ps, index, "v_scale")
        return s[0], s[1], s[2], pages, ps, heads, D, BL_DTYPE_I8
    if dtype is not torch.bfloat16:
        raise ValueError(f"k_cache: dtype must be bfloat16 or int8, got {dtype}")
    if k_scale is not None or v_scale is not None:
        raise ValueError("k_scale, v_scale: only for int8 caches")
    return s[0], s[1], s[2], pages, ps, heads, D, BL_DTYPE_BF16


def rope_append(q, k, v, pos, table, k_cache, v_cache, blocks, seq=None, k_scale=None, v_scale=None,
                interleaved: bool = False, dtype=None, out=None):
    """Rotary positions on a step's queries and keys, keys and values into a paged cache.

    q [T][q_heads][D], k and v [T][heads][D] (one dtype, any token and head strides); caches
    [pages][heads][page_size][D] in bf16, or int8 with fp32 scales [pages][heads][page_size].  Token
    t is sequence seq[t]'s (int32; None: sequence t) at position pos[t] (int32; below 0: padding);
    its page is blocks[seq][pos // page_size] (int32 [seqs][blocks per sequence]).  Returns the
    rotated queries, in ``dtype`` (that of q); ``out`` may supply them.
    """
    import torch
    if len(q.shape) != 3:
        raise ValueError(f"q: must be [T][heads][D], got {tuple(q.shape)}")
    T, _, D = q.shape
    xdt = q.dtype
    ix = _device(q, "q")
    cache = _cache_check(k_cache, v_cache, k_scale, v_scale, ix)
    positions, R = _table(table, ix)
    _buf(pos, torch.int32, T, ix, "pos")
    if len(blocks.shape) != 2:
        raise ValueError("blocks: must be [seqs][blocks per sequence]")
    seqs, per = blocks.shape
    _buf(blocks, torch.int32, 1, ix, "blocks")
    if seq is not None:
        _buf(seq, torch.int32, T, ix, "seq")
    if dtype is None:
        dtype = xdt if out is None else out.dtype
    xd, qd = _dt(xdt, "q"), _dt(dtype, "dtype")
    qt, qh, nq = _heads(q, T, D, ix, "q", xdt)
    kt, kh, nk = _heads(k, T, D, ix, "k", xdt)
    vt, vh, nv = _heads(v, T, D, ix, "v", xdt)
    if out is None:
        ot, oh, no = nq * D, D, nq
    else:
        ot, oh, no = _heads(out, T, D, ix, "out", dtype)
    heads = cache[5]
    if no != nq or nk != heads or nv != heads or D != cache[6]:
        raise ValueError("heads or head dimension of out, k, v and the cache do not fit")
    if out is None:
        out = _like(q, dtype)
    arr = _ROPE3.pack(q.data_ptr(), out.data_ptr(), qt, qh, ot, oh, nq, k.data_ptr(), 0, kt, kh, 0, 0,
                      nk, v.data_ptr(), 0, vt, vh, 0, 0, nv)
    _enqueue(ix, "bitlinear_rope_append", _lib().bitlinear_rope_append, arr, T, R, interleaved, xd,
             qd, pos.data_ptr(), _ptr(seq), blocks.data_ptr(), seqs, per, table.data_ptr(), positions,
             _KV.pack(k_cache.data_ptr(), v_cache.data_ptr(), 0 if k_scale is None else
             k_scale.data_ptr(), 0 if v_scale is None else v_scale.data_ptr(), *cache))
    return out


class PagedAttn:
    """Decode attention over a paged cache: ``PagedAttn(B, q_heads, heads, D, page_size, max_len)``
    sizes the launch and holds its workspace; calling it attends one query token per sequence.

    max_len is the length to be expected of the sequences, by which the launch is sized (longer ones are
    computed as well, on too few workgroups); window > 0 attends the last ``window`` positions only.
    Calls of one object are ordered on one stream.  Build
    it outside any graph capture (it waits for its workspace).
    """

    def __init__(self, B: int, q_heads: int, heads: int, D: int, page_size: int, max_len: int,
                 window: int = 0, device="cuda"):
        import torch
        st, self.plan = bitlinear_paged_attn_plan(B, q_heads, heads, D, max_len, window)
        _check(st, "bitlinear_paged_attn_plan")
        self.page_size = page_size
        self.shape = torch.Size((B, q_heads, D))
        self.scale = D ** -0.5
        self.ws = torch.zeros(self.plan.ws_bytes, dtype=torch.uint8, device=device)
        if self.ws.is_cuda:                 # zeroed before a call on any stream
            torch.cuda.current_stream(self.ws.device).synchronize()

    def __call__(self, q, k_cache, v_cache, blocks, lens, scale=None, k_scale=None, v_scale=None,
                 out=None, want_lse: bool = False, lse=None):
        """q [B][q_heads][D] fp32 or bf16; blocks int32 [B][blocks per sequence]; lens int32 [B].

        Returns out [B][q_heads][D] in q's dtype, or (out, lse fp32 [B][q_heads]) if lse is wanted
        or given.  scale: D ** -0.5 by default.  ``out`` and ``lse`` may supply buffers.
        """
        import torch
        ws, shape = self.ws, self.shape
        B, heads, D = shape
        ix = _device(ws, "workspace")
        if q.shape != shape:
            raise ValueError(f"q: must be {tuple(shape)}, got {tuple(q.shape)}")
        dtype = q.dtype
        qd = _dt(dtype, "q")
        qt, qh, _ = _heads(q, B, D, ix, "q", dtype)
        cache = _cache_check(k_cache, v_cache, k_scale, v_scale, ix)
        if cache[4] != self.page_size:
            raise ValueError(f"k_cache: page size must be {self.page_size}, got {cache[4]}")
        if len(blocks.shape) != 2 or blocks.shape[0] != B:
            raise ValueError(f"blocks: must be [{B}][blocks per sequence]")
        _buf(blocks, torch.int32, 0, ix, "blocks")
        _buf(lens, torch.int32, B, ix, "lens")
        if out is not None:
            _buf(out, dtype, B * heads * D, ix, "out")
        if lse is not None:
            _buf(lse, torch.float32, B * heads, ix, "lse")
        elif want_lse:
            lse = q.new_empty((B, heads), dtype=torch.float32)
        if out is None:
            out = _like(q, dtype)
        _enqueue(
            ix, "bitlinear_paged_attn", _lib().bitlinear_paged_attn,
            self.plan, q.data_ptr(), qd, qt, qh, self.scale if scale is None else scale,
            _KV.pack(k_cache.data_ptr(), v_cache.data_ptr(),
                     0 if k_scale is None else k_scale.data_ptr(),
                     0 if v_scale is None else v_scale.data_ptr(), *cache),
            blocks.data_ptr(), blocks.shape[1], lens.data_ptr(), out.data_ptr(), _ptr(lse),
            ws.data_ptr(), ws.numel())
        return out if lse is None else (out, lse)
