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

from . import bitlinear as _B
from .bitlinear import BL_DTYPE_BF16, BL_DTYPE_F32, _check, _need, _ptr, _stream

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
                ("window", ctypes.c_int32), ("splits", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("ws_bytes", _SZ)]


_fns = None


def _lib():
    """The library, with these calls' argument types declared."""
    global _fns
    if _fns is None:
        L = _B.lib()
        rd, kv, pl = (ctypes.POINTER(BlRopeDesc), ctypes.POINTER(BlKvCache),
                      ctypes.POINTER(BlAttnPlan))
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
                                        seqs, blocks_per_seq, table, positions, kv, stream)


def bitlinear_paged_attn_plan(B, q_heads, kv_heads, head_dim, max_len, window):
    """Returns (status, BlAttnPlan)."""
    plan = BlAttnPlan()
    st = _lib().bitlinear_paged_attn_plan(B, q_heads, kv_heads, head_dim, max_len, window,
                                          ctypes.byref(plan))
    return st, plan


def bitlinear_paged_attn(plan, q, q_dtype, q_tok, q_head, scale, kv, blocks, blocks_per_seq, lens,
                         out, lse, ws, ws_bytes, stream) -> int:
    return _lib().bitlinear_paged_attn(plan, q, q_dtype, q_tok, q_head, scale, kv, blocks,
                                       blocks_per_seq, lens, out, lse, ws, ws_bytes, stream)


# ---------------------------------------------------------------------------------------------
# torch convenience wrappers
# ---------------------------------------------------------------------------------------------

def _dt(dtype, name: str) -> int:
    import torch
    if dtype == torch.float32:
        return BL_DTYPE_F32
    if dtype == torch.bfloat16:
        return BL_DTYPE_BF16
    raise ValueError(f"{name}: dtype must be float32 or bfloat16, got {dtype}")


def _need2(t, T: int, K: int, device, name: str, dtype=None) -> int:
    """A contiguous [T][K] tensor; returns its dtype code."""
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name}: must be a CUDA tensor on {device}, got {t.device}")
    if tuple(t.shape) != (T, K) or not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous [{T}][{K}], got {tuple(t.shape)}")
    return _dt(t.dtype, name)


def norm_quant(x, weight=None, residual=None, eps: float = 1e-6, lift_M: int = 0,
               want_rstd: bool = False, out=None):
    """Residual addition, RMS norm and per-token int8 quantization of x[T][K] (fp32 or bf16).

    h = x + residual in residual's dtype; the normed rows h * rstd * weight (fp32 weight[K]) are
    quantized as ``act_quant(..., lift_M)`` would.  Returns (xq int8 [T][K_eff], scale fp32 [T], h,
    rstd); h is x itself without a residual, rstd (fp32 [T], for ``norm_quant_bwd``) is None unless
    wanted.  ``out`` may supply (xq, scale, h, rstd); its h may be ``residual`` (in place), or None
    without a residual.
    """
    import torch
    if x.dim() != 2:
        raise ValueError(f"x: must be [T][K], got {tuple(x.shape)}")
    T, K = x.shape
    dev = x.device
    xd = _need2(x, T, K, dev, "x")
    rd = 0 if residual is None else _need2(residual, T, K, dev, "residual")
    if weight is not None:
        _need(weight, torch.float32, K, dev, "weight")
    ke = K // lift_M * (2 * lift_M - 4) if lift_M else K
    if out is None:
        xq = torch.empty((T, ke), dtype=torch.int8, device=dev)
        scale = torch.empty(T, dtype=torch.float32, device=dev)
        h = None if residual is None else torch.empty_like(residual)
        rstd = torch.empty(T, dtype=torch.float32, device=dev) if want_rstd else None
    else:
        xq, scale, h, rstd = out
        _need(xq, torch.int8, T * ke, dev, "xq")
        _need(scale, torch.float32, T, dev, "scale")
        if (h is None) != (residual is None):
            raise ValueError("h: given exactly with a residual")
        if h is not None:
            _need2(h, T, K, dev, "h", residual.dtype)
        if rstd is not None:
            _need(rstd, torch.float32, T, dev, "rstd")
    _check(bitlinear_norm_quant(x.data_ptr(), xd, _ptr(residual), rd, _ptr(weight), eps, T, K,
                                lift_M, _ptr(h), xq.data_ptr(), scale.data_ptr(), _ptr(rstd),
                                _stream()), "bitlinear_norm_quant")
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
    if dn.dim() != 2:
        raise ValueError(f"dn: must be [T][K], got {tuple(dn.shape)}")
    T, K = dn.shape
    dev = dn.device
    gd = _need2(dn, T, K, dev, "dn")
    hd = _need2(h, T, K, dev, "h")
    _need(rstd, torch.float32, T, dev, "rstd")
    if weight is not None:
        _need(weight, torch.float32, K, dev, "weight")
    if dtype is None:
        dtype = dn.dtype if dres is None else dres.dtype
    if dres is not None:
        _need2(dres, T, K, dev, "dres", dtype)
    if out is None:
        dh = torch.empty((T, K), dtype=dtype, device=dev)
        dw = torch.empty(K, dtype=torch.float32, device=dev) if want_dw else None
    else:
        dh, dw = out
        _need2(dh, T, K, dev, "dh", dtype)
        if dw is not None:
            _need(dw, torch.float32, K, dev, "dw")
    wsb = 0
    if dw is not None:
        st, wsb = bitlinear_norm_quant_bwd_workspace_bytes(T, K)
        _check(st, "bitlinear_norm_quant_bwd_workspace_bytes")
        if ws is None:
            ws = torch.empty(wsb, dtype=torch.uint8, device=dev)
        _need(ws, torch.uint8, wsb, dev, "ws")
        wsb = ws.numel()
    _check(bitlinear_norm_quant_bwd(dn.data_ptr(), gd, h.data_ptr(), hd, rstd.data_ptr(),
                                    _ptr(weight), _ptr(dres), dh.data_ptr(), _dt(dtype, "dtype"),
                                    _ptr(dw), T, K, _ptr(ws) if dw is not None else None, wsb,
                                    _stream()), "bitlinear_norm_quant_bwd")
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
    _need(freq, torch.float64, 1, freq.device, "freq")
    half = freq.numel()
    if out is None:
        out = torch.empty((positions, half, 2), dtype=torch.float32, device=freq.device)
    _need(out, torch.float32, positions * half * 2, freq.device, "out")
    _check(bitlinear_rope_table(freq.data_ptr(), half, positions, mscale, out.data_ptr(),
                                _stream()), "bitlinear_rope_table")
    return out


def _heads(t, T: int, D: int, device, name: str, dtype=None):
    """Checks of a [T][heads][D] tensor (any strides but the last)."""
    if t.dim() != 3 or t.shape[0] != T or t.shape[2] != D:
        raise ValueError(f"{name}: must be [{T}][heads][{D}], got {tuple(t.shape)}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name}: must be a CUDA tensor on {device}, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype must be {dtype}, got {t.dtype}")
    if t.stride(2) != 1 and D > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.stride()


def _table(table, device):
    import torch
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError(f"table: must be [positions][pairs][2], got {tuple(table.shape)}")
    _need(table, torch.float32, 0, device, "table")
    return table.shape[0], 2 * table.shape[1]


def rope(xs, pos, table, interleaved: bool = False, inverse: bool = False, dtype=None, outs=None):
    """Rotary positions on up to four tensors [T][heads][D] (one dtype, any token and head strides)
    in one launch; the first 2 * table.shape[1] elements of each head are rotated.

    pos: int32 [T]; table: ``rope_table``'s.  ``inverse`` turns back, which is the gradient.
    Returns a list of tensors in ``dtype`` (that of xs); ``outs`` may supply them, and may be xs
    itself (in place).
    """
    import torch
    if not xs or xs[0].dim() != 3:
        raise ValueError("xs: must be tensors [T][heads][D]")
    T, _, D = xs[0].shape
    dev, xdt = xs[0].device, xs[0].dtype
    positions, R = _table(table, dev)
    _need(pos, torch.int32, T, dev, "pos")
    if dtype is None:
        dtype = xdt if outs is None else outs[0].dtype
    if outs is None:
        outs = [torch.empty(x.shape, dtype=dtype, device=dev) for x in xs]
    elif len(outs) != len(xs):
        raise ValueError("outs: one per tensor")
    strides = []
    for i, (x, y) in enumerate(zip(xs, outs)):
        sx = _heads(x, T, D, dev, f"xs[{i}]", xdt)
        sy = _heads(y, T, D, dev, f"outs[{i}]", dtype)
        if x.shape[1] != y.shape[1]:
            raise ValueError(f"outs[{i}]: heads differ from xs[{i}]")
        strides.append((sx[0], sx[1], sy[0], sy[1], x.shape[1]))
    arr = (BlRopeDesc * len(xs))(*(BlRopeDesc(x.data_ptr(), y.data_ptr(), *s)
                                   for x, y, s in zip(xs, outs, strides)))
    _check(bitlinear_rope(arr, T, D, R, interleaved, inverse, _dt(xdt, "xs"), _dt(dtype, "dtype"),
                          pos.data_ptr(), table.data_ptr(), positions, _stream()), "bitlinear_rope")
    return outs


def _cache_check(k, v, k_scale, v_scale, device):
    """Checks of a cache's tensors [pages][heads][page_size][D] (any strides but the last, the same
    for both) and scales [pages][heads][page_size]; returns the shape."""
    import torch
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
        raise ValueError("k_cache, v_cache: must be [pages][heads][page_size][D] with the same "
                         "shape, strides and dtype")
    if not k.is_cuda or k.device != device or v.device != device:
        raise ValueError(f"k_cache, v_cache: must be CUDA tensors on {device}")
    pages, heads, ps, D = shape = k.shape
    if k.stride(3) != 1 and D > 1:
        raise ValueError("k_cache: the last dimension must be contiguous")
    if k.dtype == torch.int8:
        _need(k_scale, torch.float32, pages * heads * ps, device, "k_scale")
        _need(v_scale, torch.float32, pages * heads * ps, device, "v_scale")
    elif k.dtype != torch.bfloat16:
        raise ValueError(f"k_cache: dtype must be bfloat16 or int8, got {k.dtype}")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale, v_scale: only for int8 caches")
    return shape


def _cache(k, v, k_scale, v_scale) -> BlKvCache:
    pages, heads, ps, D = k.shape
    s = k.stride()
    return BlKvCache(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), s[0], s[1], s[2], pages,
                     ps, heads, D, BL_DTYPE_BF16 if k_scale is None else BL_DTYPE_I8)


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
    if q.dim() != 3:
        raise ValueError(f"q: must be [T][heads][D], got {tuple(q.shape)}")
    T, _, D = q.shape
    dev, xdt = q.device, q.dtype
    _, heads, _, cache_D = _cache_check(k_cache, v_cache, k_scale, v_scale, dev)
    positions, R = _table(table, dev)
    _need(pos, torch.int32, T, dev, "pos")
    if blocks.dim() != 2:
        raise ValueError("blocks: must be [seqs][blocks per sequence]")
    _need(blocks, torch.int32, 1, dev, "blocks")
    seqs, per = blocks.shape
    if seq is not None:
        _need(seq, torch.int32, T, dev, "seq")
    if dtype is None:
        dtype = xdt if out is None else out.dtype
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=dev)
    sq, so = _heads(q, T, D, dev, "q", xdt), _heads(out, T, D, dev, "out", dtype)
    sk, sv = _heads(k, T, D, dev, "k", xdt), _heads(v, T, D, dev, "v", xdt)
    if out.shape[1] != q.shape[1] or k.shape[1] != heads or v.shape[1] != heads or D != cache_D:
        raise ValueError("heads or head dimension of out, k, v and the cache do not fit")
    arr = (BlRopeDesc * 3)(
        BlRopeDesc(q.data_ptr(), out.data_ptr(), sq[0], sq[1], so[0], so[1], q.shape[1]),
        BlRopeDesc(k.data_ptr(), None, sk[0], sk[1], 0, 0, heads),
        BlRopeDesc(v.data_ptr(), None, sv[0], sv[1], 0, 0, heads))
    _check(bitlinear_rope_append(arr, T, R, interleaved, _dt(xdt, "q"), _dt(dtype, "dtype"),
                                 pos.data_ptr(), _ptr(seq), blocks.data_ptr(), seqs, per,
                                 table.data_ptr(), positions,
                                 _cache(k_cache, v_cache, k_scale, v_scale), _stream()),
           "bitlinear_rope_append")
    return out


class PagedAttn:
    """Decode attention over a paged cache: ``PagedAttn(B, q_heads, heads, D, page_size, max_len)``
    plans the split and holds the workspace; calling it attends one query token per sequence.

    max_len is the length the split is tuned for (an upper bound of the sequences'); window > 0
    attends the last ``window`` positions only.  Calls of one object are ordered on one stream.
    """

    def __init__(self, B: int, q_heads: int, heads: int, D: int, page_size: int, max_len: int,
                 window: int = 0, device="cuda"):
        import torch
        st, self.plan = bitlinear_paged_attn_plan(B, q_heads, heads, D, max_len, window)
        _check(st, "bitlinear_paged_attn_plan")
        self.page_size = page_size
        self.ws = torch.zeros(self.plan.ws_bytes, dtype=torch.uint8, device=device)

    def __call__(self, q, k_cache, v_cache, blocks, lens, scale=None, k_scale=None, v_scale=None,
                 out=None, want_lse: bool = False, lse=None):
        """q [B][q_heads][D] fp32 or bf16; blocks int32 [B][blocks per sequence]; lens int32 [B].

        Returns out [B][q_heads][D] in q's dtype, or (out, lse fp32 [B][q_heads]) if lse is wanted
        or given.  scale: D ** -0.5 by default.  ``out`` and ``lse`` may supply buffers.
        """
        import torch
        p, dev = self.plan, self.ws.device
        if tuple(q.shape) != (p.B, p.q_heads, p.head_dim):
            raise ValueError(f"q: must be [{p.B}][{p.q_heads}][{p.head_dim}], got {tuple(q.shape)}")
        s = _heads(q, p.B, p.head_dim, dev, "q")
        qd = _dt(q.dtype, "q")
        page = _cache_check(k_cache, v_cache, k_scale, v_scale, dev)[2]
        if page != self.page_size:
            raise ValueError(f"k_cache: page size must be {self.page_size}, got {page}")
        if blocks.dim() != 2 or blocks.shape[0] != p.B:
            raise ValueError(f"blocks: must be [{p.B}][blocks per sequence]")
        _need(blocks, torch.int32, 0, dev, "blocks")
        _need(lens, torch.int32, p.B, dev, "lens")
        if out is None:
            out = torch.empty((p.B, p.q_heads, p.head_dim), dtype=q.dtype, device=dev)
        else:
            _need(out, q.dtype, p.B * p.q_heads * p.head_dim, dev, "out")
        if lse is not None:
            _need(lse, torch.float32, p.B * p.q_heads, dev, "lse")
        elif want_lse:
            lse = torch.empty((p.B, p.q_heads), dtype=torch.float32, device=dev)
        _check(bitlinear_paged_attn(p, q.data_ptr(), qd, s[0], s[1],
                                    p.head_dim ** -0.5 if scale is None else scale,
                                    _cache(k_cache, v_cache, k_scale, v_scale), blocks.data_ptr(), blocks.shape[1], lens.data_ptr(),
                                    out.data_ptr(), _ptr(lse), self.ws.data_ptr(), p.ws_bytes,
                                    _stream()), "bitlinear_paged_attn")
        return out if lse is None else (out, lse)
