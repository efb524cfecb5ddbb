"""Cases and plain forms of the operators around the BitLinear projections of a decoder block.

Five operators, in the order a block runs them:

  norm        the residual's addition, root-mean-square norm and per-token int8 quantization that
              feed a projection (``norm_quant``)
  norm_bwd    its gradient (``norm_quant_bwd``)
  rope        rotary positions on the heads of several tensors, and their inverse, the gradient
              (``rope``)
  append      rotary positions on a step's queries and keys, keys and values written into a paged
              cache in bf16 or int8 (``rope_append``)
  attn        attention of one new token per sequence over that cache (``PagedAttn``)

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or, with
``own`` set, by the calls a user of the library makes.  Two plain steps are spelled so that the
int8 values are those of the definition: the mean square is summed in 64 bits (the definition's
sum, so that the order of the sum cannot move a value across a rounding boundary), and divisions
are written with tensor divisors (torch multiplies by a reciprocal otherwise, which is not the
correctly rounded quotient).
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2, "i8": 1, "none": 0}


def _lib():
    import sparsity_amd
    return sparsity_amd


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # One decode step's smallest call: one token entering a projection of 2560 features.  The
        # projection's fp32 output is added to a bf16 residual stream.  Latency is all it costs.
        {"name": "norm_decode", "op": "norm", "T": 1, "K": 2560, "x": "f32", "res": "bf16",
         "lift": 0, "train": False},
        # A prompt of 2048 tokens in front of a 6:8 projection (lifted int8 rows), with an fp32
        # residual stream.
        {"name": "norm_prompt_lift", "op": "norm", "T": 2048, "K": 4096, "x": "bf16", "res": "f32",
         "lift": 8, "train": False},
        # The norm of a training step of the 3200-wide layer set at 8192 tokens.
        {"name": "norm_train", "op": "norm", "T": 8192, "K": 3200, "x": "f32", "res": "bf16",
         "lift": 0, "train": True},
        # The backward of the same norm: the fp32 gradient of the projections' input, the residual
        # stream's gradient joining it.
        {"name": "norm_train_back", "op": "norm_bwd", "T": 8192, "K": 3200, "dn": "f32",
         "h": "bf16", "grad": "bf16", "dres": True},
        # Rotary positions on a training step's queries and keys (25 heads of 128 each), half
        # layout, from the projections' fp32 outputs to bf16.
        {"name": "rope_train", "op": "rope", "T": 8192, "Hq": 25, "Hk": 25, "D": 128, "R": 128,
         "inter": False, "inverse": False, "x": "f32", "y": "bf16", "fused": False},
        # The gradient through rotary positions on part of the head, interleaved layout, on the
        # slices of a fused query-key-value buffer, at an odd number of tokens.
        {"name": "rope_back_partial", "op": "rope", "T": 1021, "Hq": 32, "Hk": 8, "D": 80, "R": 32,
         "inter": True, "inverse": True, "x": "bf16", "y": "bf16", "fused": True},
        # A decode step's queries, keys and values for 16 sequences (20 heads, 5 of them for keys
        # and values) entering a bf16 cache with pages of 16 tokens.
        {"name": "append_decode", "op": "append", "T": 16, "Hq": 20, "Hk": 5, "D": 128, "R": 128,
         "inter": False, "x": "f32", "q": "bf16", "kv": "bf16", "page": 16, "seqs": 16,
         "ctx": 1536},
        # A prompt of 4096 tokens entering an int8 cache with pages of 64 tokens.
        {"name": "append_prompt_int8", "op": "append", "T": 4096, "Hq": 32, "Hk": 8, "D": 128,
         "R": 128, "inter": False, "x": "f32", "q": "bf16", "kv": "i8", "page": 64, "seqs": 1,
         "ctx": 4096},
        # One sequence of 700 tokens: the smallest attention call, fp32 queries and output.
        {"name": "attn_short", "op": "attn", "B": 1, "Hq": 20, "Hk": 5, "D": 128, "len": 700,
         "ragged": False, "page": 16, "kv": "bf16", "q": "f32", "window": 0},
        # A serving batch of 48 ragged sequences (an empty one and one of a single token among
        # them) over an int8 cache.
        {"name": "attn_ragged_int8", "op": "attn", "B": 48, "Hq": 32, "Hk": 8, "D": 128,
         "len": 6001, "ragged": True, "page": 32, "kv": "i8", "q": "bf16", "window": 0},
        # A full batch: 64 sequences of 8192 tokens, 2 GB of bf16 cache.
        {"name": "attn_batch", "op": "attn", "B": 64, "Hq": 32, "Hk": 8, "D": 128, "len": 8192,
         "ragged": False, "page": 16, "kv": "bf16", "q": "bf16", "window": 0},
        # One sequence with a very long context: few rows, one long axis.
        {"name": "attn_long", "op": "attn", "B": 1, "Hq": 20, "Hk": 5, "D": 128, "len": 262144,
         "ragged": False, "page": 64, "kv": "bf16", "q": "bf16", "window": 0},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    v = max(lo, min(hi, int(v / step) * step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rope", "append", "attn", "attn"])
    if op == "norm":
        lift = rng.choice([0, 0, 0, 8, 16])
        K = _log(rng, 64, 16384, max(8, lift))
        return {"op": op, "T": _log(rng, 1, min(8192, (32 << 20) // K)), "K": K,
                "x": rng.choice(["f32", "bf16"]), "res": rng.choice(["f32", "bf16", "none"]),
                "lift": lift, "train": rng.random() < 0.5}
    if op == "norm_bwd":
        K = _log(rng, 64, 16384, 8)
        return {"op": op, "T": _log(rng, 1, min(8192, (32 << 20) // K)), "K": K,
                "dn": rng.choice(["f32", "bf16"]), "h": rng.choice(["f32", "bf16"]),
                "grad": rng.choice(["f32", "bf16"]), "dres": rng.random() < 0.7}
    D = rng.choice([64, 80, 96, 128, 128, 256])
    Hk = rng.choice([1, 2, 5, 8, 25])
    if op == "rope":
        Hq = Hk * rng.choice([1, 2, 4])
        return {"op": op, "T": _log(rng, 1, min(8192, (32 << 20) // ((Hq + Hk) * D))), "Hq": Hq,
                "Hk": Hk, "D": D, "R": rng.choice([D, D, D // 2]), "inter": rng.random() < 0.5,
                "inverse": rng.random() < 0.5, "x": rng.choice(["f32", "bf16"]),
                "y": rng.choice(["f32", "bf16"]), "fused": rng.random() < 0.5}
    if op == "append":
        Hq = Hk * rng.choice([1, 2, 4, 8])
        seqs = _log(rng, 1, 64)
        T = seqs if rng.random() < 0.5 else min(4096, seqs * _log(rng, 1, 512))
        T = max(T, seqs)
        ctx = -(-T // seqs) + _log(rng, 1, max(1, min(2048, 65536 // seqs)))
        return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": rng.choice([D, D, D // 2]),
                "inter": rng.random() < 0.5, "x": rng.choice(["f32", "bf16"]),
                "q": rng.choice(["f32", "bf16"]), "kv": rng.choice(["bf16", "i8"]),
                "page": rng.choice([1, 8, 16, 24, 64]), "seqs": seqs, "ctx": ctx + (ctx == 3072)}
    B = _log(rng, 1, 64)
    most = 400_000_000 // (B * Hk * D)
    return {"op": op, "B": B, "Hq": Hk * rng.choice([1, 2, 4, 5, 8, 16, 20]), "Hk": Hk, "D": D,
            "len": _log(rng, 1, min(131072, most)), "ragged": B > 3 and rng.random() < 0.7,
            "page": rng.choice([1, 8, 16, 24, 64, 256]), "kv": rng.choice(["bf16", "i8"]),
            "q": rng.choice(["f32", "bf16"]), "window": rng.choice([0, 0, 0, 500])}


def _keff(c):
    return c["K"] // c["lift"] * (2 * c["lift"] - 4) if c["lift"] else c["K"]


def _lens(c):
    """The sequences' lengths, in an order that the seed shuffles: all of them `len`, or ragged
    ones from none and one upwards."""
    if not c["ragged"]:
        return [c["len"]] * c["B"]
    return [0, 1, c["len"]] + [1 + int(c["len"] * (i * 0.6180339887 % 1.0))
                               for i in range(3, c["B"])]


def _attended(c):
    return [min(n, c["window"]) if c["window"] else n for n in _lens(c)]


def _pages(c):
    """Pages per sequence and pages in all, some of them free."""
    per = -(-(c["len"] if c["op"] == "attn" else c["ctx"]) // c["page"])
    return per, per * (c["B"] if c["op"] == "attn" else c["seqs"]) + 3


def work(c):
    op = c["op"]
    if op == "norm":
        n = c["T"] * c["K"]
        b = n * (BYTES[c["x"]] + 2 * BYTES[c["res"]]) + c["T"] * _keff(c) + 4 * c["K"] + \
            c["T"] * (8 if c["train"] else 4)
        return {"bytes": b, "flops": 8 * n}
    if op == "norm_bwd":
        n = c["T"] * c["K"]
        b = n * (BYTES[c["dn"]] + BYTES[c["h"]] + BYTES[c["grad"]] * (1 + c["dres"])) + \
            8 * c["K"] + 4 * c["T"]
        return {"bytes": b, "flops": 10 * n}
    if op == "rope":
        n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": n * (BYTES[c["x"]] + BYTES[c["y"]]) + c["T"] * (4 * c["R"] + 4),
                "flops": 3 * n}
    if op == "append":
        q, kv = c["T"] * c["Hq"] * c["D"], 2 * c["T"] * c["Hk"] * c["D"]
        s = 8 * c["T"] * c["Hk"] if c["kv"] == "i8" else 0
        return {"bytes": (q + kv) * BYTES[c["x"]] + q * BYTES[c["q"]] + kv * BYTES[c["kv"]] + s +
                c["T"] * (4 * c["R"] + 12), "flops": 3 * (q + kv)}
    keys = sum(_attended(c))
    kv = 2 * keys * c["Hk"] * c["D"] * BYTES[c["kv"]] + (8 * keys * c["Hk"] if c["kv"] == "i8" else 0)
    return {"bytes": kv + 2 * c["B"] * c["Hq"] * c["D"] * BYTES[c["q"]] + 4 * c["B"] * c["Hq"] +
            4 * sum(-(-n // c["page"]) for n in _attended(c)),
            "flops": 4 * keys * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _table(positions, R, dev):
    """cos and sin of position * 10000^(-2i/R), [positions][R/2][2], each rounded once to 32 bits."""
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)
    a = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float()


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype="f32", std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(DTYPES[dtype])

    op, s = c["op"], {"case": c}
    if op == "norm":
        s["x"] = normal(c["T"], c["K"], dtype=c["x"])
        s["res"] = None if c["res"] == "none" else normal(c["T"], c["K"], dtype=c["res"], std=3.0)
        s["w"] = 1.0 + normal(c["K"], std=0.1)
        return s
    if op == "norm_bwd":
        s["dn"] = normal(c["T"], c["K"], dtype=c["dn"], std=2.0 ** -10)
        s["h"] = normal(c["T"], c["K"], dtype=c["h"], std=3.0)
        s["rstd"] = (s["h"].float().square().mean(-1) + EPS).rsqrt()   # the forward kept it
        s["w"] = 1.0 + normal(c["K"], std=0.1)
        s["dres"] = normal(c["T"], c["K"], dtype=c["grad"], std=2.0 ** -10) if c["dres"] else None
        return s
    Hk, D = c["Hk"], c["D"]
    if op == "rope":
        T, Hq = c["T"], c["Hq"]
        if c["fused"]:   # queries and keys are slices of the projection's [T][(Hq + 2 Hk) D] rows
            qkv = normal(T, Hq + 2 * Hk, D, dtype=c["x"])
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = normal(T, Hq, D, dtype=c["x"]), normal(T, Hk, D, dtype=c["x"])
        s["pos"] = torch.arange(T, dtype=torch.int32, device=dev)
        s["table"] = _table(T, c["R"], dev)
        return s
    per, pages = _pages(c)
    n = c["B"] if op == "attn" else c["seqs"]
    s["blocks"] = torch.randperm(pages, generator=g, device=dev)[:n * per].view(n, per).int()
    shape = (pages, Hk, c["page"], D)   # a head's tokens of one page lie together
    if c["kv"] == "bf16":
        s["kc"], s["vc"] = (torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
                            for _ in range(2))
        s["ks"] = s["vs"] = None
    else:
        s["kc"], s["vc"] = (torch.randint(-127, 128, shape, generator=g, device=dev,
                                          dtype=torch.int8) for _ in range(2))
        s["ks"], s["vs"] = (0.01 + 0.01 * torch.rand(shape[:3], generator=g, device=dev)
                            for _ in range(2))
    if op == "append":
        T = c["T"]
        s["q"], s["k"], s["v"] = (normal(T, h, D, dtype=c["x"]) for h in (c["Hq"], Hk, Hk))
        t = torch.arange(T, device=dev)
        s["seq"] = (t % n).int()
        # each sequence's new tokens are the last ones of its context
        s["pos"] = (c["ctx"] - (T - (t % n) + n - 1) // n + t // n).int()
        s["table"] = _table(c["ctx"], c["R"], dev)
        return s
    s["q"] = normal(c["B"], c["Hq"], D, dtype=c["q"])
    s["lens"] = torch.tensor(_lens(c), device=dev, dtype=torch.int32)[
        torch.randperm(c["B"], generator=g, device=dev)].contiguous()
    if own:   # the plan holds the call's scratch memory: a program keeps it from step to step
        s["plan"] = _lib().PagedAttn(c["B"], c["Hq"], Hk, D, c["page"], c["len"], window=c["window"])
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _quant(v):
    """int8 rows and scales of v[..., K]: absmax / 127 per row, rounded half to even."""
    amax = v.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, 127.0)
    step = torch.where(amax > 0, top / amax, 0.0)
    return (v * step).round().clamp(-127, 127).to(torch.int8), (amax / top)[..., 0]


def _plain_norm(c, s):
    h = s["x"].float()
    if s["res"] is not None:
        s_res = s["res"]
        h = (h + s_res.float()).to(s_res.dtype)
    f = h.float()
    ms = (f * f).sum(-1, dtype=torch.float64) / c["K"]
    rstd = (1.0 / (ms + EPS).sqrt()).float()
    q, scale = _quant(f * rstd[:, None] * s["w"])
    if c["lift"]:
        M = c["lift"]
        q = q.view(c["T"], c["K"] // M, M).unfold(2, 4, 2).reshape(c["T"], _keff(c))
    out = {"xq": q, "scale": scale}
    if s["res"] is not None:
        out["h"] = h
    if c["train"]:
        out["rstd"] = rstd
    return out


def _plain_norm_bwd(c, s):
    h, r, g = s["h"].float(), s["rstd"][:, None], s["dn"].float()
    n = h * r
    gw = g * s["w"]
    dh = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return {"dh": dh.to(DTYPES[c["grad"]]), "dw": (g * n).sum(0)}


def _rotate(x, cs, inter, inverse):
    """x[T][H][D] in 32 bits, its first R elements of each head rotated by cs[T][R/2][2]."""
    R = 2 * cs.shape[1]
    co, si = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        si = -si
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    u, w = a * co - b * si, b * co + a * si
    y = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((y, x[..., R:]), -1)


def _plain_rope(c, s):
    cs = s["table"][s["pos"]]
    return {n: _rotate(s[n].float(), cs, c["inter"], c["inverse"]).to(DTYPES[c["y"]])
            for n in ("q", "k")}


def _plain_append(c, s):
    cs = s["table"][s["pos"]]
    q = _rotate(s["q"].float(), cs, c["inter"], False).to(DTYPES[c["q"]])
    k, v = _rotate(s["k"].float(), cs, c["inter"], False), s["v"].float()
    page = s["blocks"][s["seq"], s["pos"] // c["page"]].long()
    off = (s["pos"] % c["page"]).long()
    if c["kv"] == "bf16":
        s["kc"][page, :, off] = k.bfloat16()
        s["vc"][page, :, off] = v.bfloat16()
        return {"q": q, "kc": s["kc"], "vc": s["vc"]}
    s["kc"][page, :, off], s["ks"][page, :, off] = _quant(k)
    s["vc"][page, :, off], s["vs"][page, :, off] = _quant(v)
    return {"q": q, "kc": s["kc"], "vc": s["vc"], "ks": s["ks"], "vs": s["vs"]}


def _plain_attn(c, s):
    B, Hq, Hk, D = c["B"], c["Hq"], c["Hk"], c["D"]
    t = torch.arange(c["len"], device=s["q"].device)
    page, off = s["blocks"][:, t // c["page"]].long(), (t % c["page"]).expand(B, -1)
    k, v = s["kc"][page, :, off].float(), s["vc"][page, :, off].float()   # [B][len][Hk][D]
    if s["ks"] is not None:
        k = k * s["ks"][page, :, off][..., None]
        v = v * s["vs"][page, :, off][..., None]
    live = t < s["lens"][:, None]
    if c["window"]:
        live = live & (t >= s["lens"][:, None] - c["window"])
    live = live[:, None, None]
    q = s["q"].float().view(B, Hk, Hq // Hk, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * D ** -0.5
    score = torch.where(live, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(live, torch.exp(score - top), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3).contiguous())
    out = torch.where(total > 0, out / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return {"out": out.view(B, Hq, D).to(DTYPES[c["q"]]), "lse": lse.view(B, Hq)}


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "rope": _plain_rope,
         "append": _plain_append, "attn": _plain_attn}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return PLAIN[op](c, s)
    L = _lib()
    if op == "norm":
        xq, scale, h, rstd = L.norm_quant(s["x"], s["w"], s["res"], eps=EPS, lift_M=c["lift"],
                                          want_rstd=c["train"])
        out = {"xq": xq, "scale": scale}
        if s["res"] is not None:
            out["h"] = h
        if c["train"]:
            out["rstd"] = rstd
        return out
    if op == "norm_bwd":
        dh, dw = L.norm_quant_bwd(s["dn"], s["h"], s["rstd"], s["w"], s["dres"],
                                  dtype=DTYPES[c["grad"]])
        return {"dh": dh, "dw": dw}
    if op == "rope":
        q, k = L.rope([s["q"], s["k"]], s["pos"], s["table"], interleaved=c["inter"],
                      inverse=c["inverse"], dtype=DTYPES[c["y"]])
        return {"q": q, "k": k}
    if op == "append":
        q = L.rope_append(s["q"], s["k"], s["v"], s["pos"], s["table"], s["kc"], s["vc"],
                          s["blocks"], seq=s["seq"], k_scale=s["ks"], v_scale=s["vs"],
                          interleaved=c["inter"], dtype=DTYPES[c["q"]])
        out = {"q": q, "kc": s["kc"], "vc": s["vc"]}
        if s["ks"] is not None:
            out.update(ks=s["ks"], vs=s["vs"])
        return out
    out, lse = s["plan"](s["q"], s["kc"], s["vc"], s["blocks"], s["lens"], k_scale=s["ks"],
                         v_scale=s["vs"], want_lse=True)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_rotate(x, cs, inter, inverse):
    """Rotation as a complex product of the pairs."""
    R = 2 * cs.shape[1]
    x, cs = x.double(), cs.double()
    head = x[..., :R]
    pair = head.unflatten(-1, (R // 2, 2)) if inter else head.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    turn = torch.view_as_complex(cs.contiguous())[:, None]
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) *
                           (turn.conj() if inverse else turn))
    y = y if inter else y.transpose(-1, -2)
    return torch.cat((y.flatten(-2), x[..., R:]), -1)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "norm":
        h = s["x"].double()
        if s["res"] is not None:   # the stream is stored in its own type, and that is what is normed
            h = (h + s["res"].double()).to(s["res"].dtype).double()
        rstd = ((h ** 2).mean(-1) + EPS) ** -0.5
        n = h * rstd[:, None] * s["w"].double()
        out = {"xq": None, "scale": n.abs().amax(-1) / 127}
        if s["res"] is not None:
            out["h"] = s["x"].double() + s["res"].double()
        if c["train"]:
            out["rstd"] = rstd
        return out
    if op == "norm_bwd":   # by differentiating the norm itself; rstd is the forward's, held in 32 bits
        h = s["h"].double().requires_grad_()
        w = s["w"].double().requires_grad_()
        n = h * ((h ** 2).mean(-1, keepdim=True) + EPS) ** -0.5 * w
        dh, dw = torch.autograd.grad(n, (h, w), s["dn"].double())
        return {"dh": dh + (0 if s["dres"] is None else s["dres"].double()), "dw": dw}
    if op == "rope":
        cs = s["table"][s["pos"].long()]
        return {n: _exact_rotate(s[n], cs, c["inter"], c["inverse"]) for n in ("q", "k")}
    if op == "append":
        cs = s["table"][s["pos"].long()]
        q, k = (_exact_rotate(s[n], cs, c["inter"], False) for n in ("q", "k"))
        v = s["v"].double()
        slot = (s["blocks"][s["seq"].long(), s["pos"].long() // c["page"]].long(),
                slice(None), s["pos"].long() % c["page"])
        out = {"q": q, "kc": None, "vc": None}
        for name, x in (("k", k), ("v", v)):
            held = s[name + ("c" if c["kv"] == "bf16" else "s")].double()
            held[slot] = x if c["kv"] == "bf16" else x.abs().amax(-1) / 127
            out[name + ("c" if c["kv"] == "bf16" else "s")] = held
        return out
    B, Hq, Hk, D = c["B"], c["Hq"], c["Hk"], c["D"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == first:
            continue
        t = torch.arange(first, n, device=s["q"].device)
        page, off = s["blocks"][b, t // c["page"]].long(), t % c["page"]
        k, v = s["kc"][page, :, off].double(), s["vc"][page, :, off].double()
        if s["ks"] is not None:
            k = k * s["ks"][page, :, off].double()[..., None]
            v = v * s["vs"][page, :, off].double()[..., None]
        for j in range(Hk):
            rows = slice(j * (Hq // Hk), (j + 1) * (Hq // Hk))
            score = s["q"][b, rows].double() @ k[:, j].T / math.sqrt(D)
            lse[b, rows] = torch.logsumexp(score, -1)
            out[b, rows] = torch.softmax(score, -1) @ v[:, j]
    return {"out": out, "lse": lse}
