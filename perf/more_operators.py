"""Cases and plain forms of the operators around a model's blocks: what turns token ids into the first
block's input, the last block's output into the next token ids, and requests into a step's tables.

Five operators, in the order a step runs them:

  kv         pages and slots of a paged cache for the tokens that each request adds (``kv_step``)
  embed      rows of the embedding table by token id (``embed``)
  embed_bwd  their gradient (``embed_bwd``)
  q4         int8 rows times weights held in 4 bits with a scale per group of columns (``q4_fwd``)
  sample     temperature, top-k, top-p and min-p from one given random number per row (``sample``)

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or, with ``own``
set, by the calls a user of the library makes.  Sampling is defined on whole numbers: a token's weight
is round(2^40 exp((x - max) / temperature)), computed in 64 bits, so that no sum depends on its order
and a random number that falls next to a border still has one answer.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def _lib():
    import sparsity_amd
    return sparsity_amd


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # A decode step's tables: 64 requests add a token each, three of them have ended and give
        # their pages back.
        {"name": "kv_decode", "op": "kv", "B": 64, "page": 16, "per": 128, "T": 64, "most": 1,
         "ended": 3, "short": False},
        # Prompts entering a running batch: 500 requests add up to 256 tokens each into 65536 rows,
        # with too few free pages for all of them.
        {"name": "kv_prompts", "op": "kv", "B": 500, "page": 32, "per": 96, "T": 65536, "most": 256,
         "ended": 20, "short": True},
        # Embedding rows of a decode step of 16 sequences: latency is all it costs.
        {"name": "embed_decode", "op": "embed", "T": 16, "V": 131072, "K": 2560, "table": "bf16",
         "y": "bf16", "scaled": False, "pad": 0.0},
        # Embedding rows of a training step of the 3200-wide layer set, from fp32 masters, scaled
        # by sqrt(K); a padded batch.
        {"name": "embed_train", "op": "embed", "T": 8192, "V": 32000, "K": 3200, "table": "f32",
         "y": "bf16", "scaled": True, "pad": 0.1},
        # The gradient of that step, written over a table's gradient: most rows get no token.
        {"name": "embed_back", "op": "embed_bwd", "T": 8192, "V": 32000, "K": 3200, "dy": "bf16",
         "scaled": True, "accum": False, "ids": "zipf", "pad": 0.1},
        # The gradient of a larger step added to what a tied output head has left in the table's
        # gradient, at an odd number of tokens.
        {"name": "embed_back_tied", "op": "embed_bwd", "T": 32749, "V": 131072, "K": 2560,
         "dy": "f32", "scaled": False, "accum": True, "ids": "zipf", "pad": 0.0},
        # A projection of 6912 features in one decode step of 4 sequences.
        {"name": "q4_projection", "op": "q4", "T": 4, "n": 2560, "K": 6912, "group": 32},
        # The output head of one sequence: 131072 tokens from 2560 features.
        {"name": "q4_head", "op": "q4", "T": 1, "n": 131072, "K": 2560, "group": 64},
        # An output head of an odd number of tokens for a batch of 16.
        {"name": "q4_head_16", "op": "q4", "T": 16, "n": 100003, "K": 4096, "group": 128},
        # The largest batch: 64 sequences.
        {"name": "q4_head_64", "op": "q4", "T": 64, "n": 131072, "K": 2560, "group": 64},
        # One sequence's next token, top-k 50 and top-p 0.9.
        {"name": "sample_one", "op": "sample", "B": 1, "V": 131072, "x": "f32", "std": 2.5,
         "temp": 0.8, "k": 50, "p": 0.9, "min_p": 0.0, "mixed": False, "masked": 0.0},
        # A serving batch: 64 requests, each with its own settings (greedy, unfiltered, top-k,
        # top-p, min-p), some tokens masked.
        {"name": "sample_batch", "op": "sample", "B": 64, "V": 131072, "x": "f32", "std": 2.5,
         "temp": 1.0, "k": 0, "p": 1.0, "min_p": 0.0, "mixed": True, "masked": 0.05},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["kv", "embed", "embed_bwd", "q4", "q4", "sample", "sample"])
    if op == "kv":
        B = _log(rng, 1, 4096)
        most = rng.choice([1, 1, 5, 100, 1000])
        page = rng.choice([1, 8, 16, 24, 64])
        per = min(max(2, -(-2 * most // page)) + _log(rng, 1, 64), (1 << 22) // B)
        T = min(65536, max(1, B * most // rng.choice([1, 1, 2, 3])))
        return {"op": op, "B": B, "page": page, "per": per, "T": T, "most": most,
                "ended": rng.randrange(0, 1 + B // 8), "short": rng.random() < 0.4}
    if op == "embed":
        K = _log(rng, 64, 16384, 8)
        return {"op": op, "T": _log(rng, 1, min(16384, (64 << 20) // K)),
                "V": _log(rng, 16, min(262144, (320 << 20) // K)), "K": K,
                "table": rng.choice(["f32", "bf16"]), "y": rng.choice(["f32", "bf16"]),
                "scaled": rng.random() < 0.5, "pad": rng.choice([0.0, 0.0, 0.2])}
    if op == "embed_bwd":
        K = _log(rng, 64, 8192, 8)
        return {"op": op, "T": _log(rng, 1, min(32768, (64 << 20) // K)),
                "V": _log(rng, 16, min(131072, (300 << 20) // K)), "K": K,
                "dy": rng.choice(["f32", "bf16"]), "scaled": rng.random() < 0.5,
                "accum": rng.random() < 0.5, "ids": rng.choice(["zipf", "zipf", "even", "one"]),
                "pad": rng.choice([0.0, 0.0, 0.3])}
    if op == "q4":
        group = rng.choice([32, 64, 128])
        K = _log(rng, 128, 16384, group)
        return {"op": op, "T": rng.choice([1, _log(rng, 1, 64)]),
                "n": _log(rng, 16, min(131072, (320 << 20) // K)), "K": K, "group": group}
    B = _log(rng, 1, 64)
    V = _log(rng, 2, min(262144, (8 << 20) // B))
    return {"op": op, "B": B, "V": V, "x": rng.choice(["f32", "bf16"]),
            "std": rng.choice([0.5, 1.0, 2.5, 5.0]), "temp": rng.choice([0.0, 0.3, 0.8, 1.0, 1.5]),
            "k": rng.choice([0, 0, 1, 40, _log(rng, 1, V)]), "p": rng.choice([1.0, 1.0, 0.5, 0.95]),
            "min_p": rng.choice([0.0, 0.0, 0.05]), "mixed": rng.random() < 0.3,
            "masked": rng.choice([0.0, 0.0, 0.5])}


def work(c):
    op = c["op"]
    if op == "kv":   # lengths in, lengths and starts out; the rows of T tokens; a page per new block
        return {"bytes": 16 * c["B"] + 16 * c["T"] + 8 * (c["T"] // c["page"] + 1),
                "flops": 4 * c["T"] + 8 * c["B"]}
    if op == "embed":
        live = int(c["T"] * (1.0 - c["pad"]))
        return {"bytes": live * c["K"] * BYTES[c["table"]] + c["T"] * (c["K"] * BYTES[c["y"]] + 4),
                "flops": live * c["K"]}
    if op == "embed_bwd":
        live = int(c["T"] * (1.0 - c["pad"]))
        rows = {"one": 1, "even": c["V"] * -math.expm1(-live / c["V"]),
                "zipf": _zipf_rows(live, c["V"])}[c["ids"]]
        out = 8 * rows * c["K"] if c["accum"] else 4 * c["V"] * c["K"]
        return {"bytes": live * c["K"] * BYTES[c["dy"]] + 4 * c["T"] + out, "flops": live * c["K"]}
    if op == "q4":
        w = c["n"] * c["K"]
        return {"bytes": w // 2 + 2 * w // c["group"] + c["T"] * (c["K"] + 4 + 4 * c["n"]),
                "flops": 2 * w * c["T"]}
    n = c["B"] * c["V"]
    return {"bytes": n * BYTES[c["x"]] + c["B"] * 32, "flops": 4 * n}


def _zipf_rows(T, V):
    """Distinct ids to be expected of T ids that are log-uniform over V."""
    rows, lo = 0.0, 1
    while lo <= V:   # sixteenths of an octave at a time
        hi = max(lo + 1, int(lo * 1.0443))
        n = min(hi, V + 1) - lo
        p = math.log((lo + n) / lo) / math.log(V + 1) / n
        rows += n * -math.expm1(T * math.log1p(-min(p, 1 - 1e-9)))
        lo += n
    return rows


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _ids(c, g, dev, kind):
    T, V = c["T"], c["V"]
    if kind == "one":
        ids = torch.full((T,), V // 2, device=dev, dtype=torch.int32)
    elif kind == "even":
        ids = torch.randint(0, V, (T,), generator=g, device=dev, dtype=torch.int32)
    else:   # a few ids make up much of a text: log-uniform ranks, in a shuffled order of the ids
        u = torch.rand(T, generator=g, device=dev, dtype=torch.float64)
        rank = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
        ids = torch.randperm(V, generator=g, device=dev)[rank].int()
    if c["pad"]:
        ids[torch.rand(T, generator=g, device=dev) < c["pad"]] = -1
    return ids


def _quantize(W, group):
    """Signed 4-bit values and bf16 scales: absmax / 7 of each group of a row, rounded to bf16; the
    quotient by that scale rounded half to even."""
    n, K = W.shape
    w = W.view(n, K // group, group)
    amax = w.abs().amax(-1)
    scales = (amax / torch.full_like(amax, 7.0)).bfloat16()
    s = scales.float()[..., None]
    q = torch.where(s > 0, (w / s).round().clamp(-7, 7), 0.0).to(torch.int8)
    return q.view(n, K), scales


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    op, s = c["op"], {"case": c}
    if op == "kv":
        B, per, page = c["B"], c["per"], c["page"]
        room = per * page
        most = min(c["most"], room)
        fresh = (rand(B) * most).int() + 1
        cached = (rand(B) * (room - most + 1)).int().clamp_(max=room - most)
        if c["most"] > 1:   # a part of the requests begins
            cached[rand(B) < 0.5] = 0
        fresh[torch.randperm(B, generator=g, device=dev)[:c["ended"]]] = -1
        pages = torch.randperm(B * per + 8, generator=g, device=dev).int()
        s["cached"], s["fresh"] = cached, fresh
        s["blocks"] = pages[:B * per].view(B, per).contiguous()
        have = (cached + page - 1) // page
        col = torch.arange(per, device=dev)
        spare = torch.where(col < have[:, None], -1, s["blocks"]).flatten()   # pages no request holds
        s["blocks"][col >= have[:, None]] = -1
        spare = torch.cat((spare[spare >= 0], pages[B * per:]))
        s["free"] = torch.full((pages.numel(),), -1, dtype=torch.int32, device=dev)
        s["free"][:spare.numel()] = spare
        n = torch.tensor([spare.numel()], dtype=torch.int32, device=dev)
        if c["short"]:   # pages for about half of what is wanted
            want = ((cached + fresh.clamp(min=0) + page - 1) // page - have).sum()
            n = torch.minimum(n, (want // 2).int())
        s["count"] = n
        return s
    if op in ("embed", "embed_bwd"):
        T, V, K = c["T"], c["V"], c["K"]
        s["scale"] = math.sqrt(K) if c["scaled"] else 1.0
        s["ids"] = _ids(c, g, dev, c.get("ids", "zipf"))
        if op == "embed":
            s["table"] = (torch.randn(V, K, generator=g, device=dev) * 0.02).to(DTYPES[c["table"]])
        else:
            s["dy"] = (torch.randn(T, K, generator=g, device=dev) * 2.0 ** -10).to(DTYPES[c["dy"]])
            if c["accum"]:
                s["dtable"] = torch.randn(V, K, generator=g, device=dev) * 2.0 ** -10
        return s
    if op == "q4":
        T, n, K = c["T"], c["n"], c["K"]
        W = torch.randn(n, K, generator=g, device=dev) * 0.02
        s["xq"] = (torch.randn(T, K, generator=g, device=dev) * 32).round_().clamp_(-127, 127).to(torch.int8)
        s["scale"] = 0.01 + 0.05 * rand(T)
        if own:   # weights are laid out once
            s["codes"], s["scales"] = _lib().q4_pack(W, c["group"])
        else:
            s["q"], s["scales"] = _quantize(W, c["group"])
        return s
    B, V = c["B"], c["V"]
    x = torch.randn(B, V, generator=g, device=dev) * c["std"]
    if c["masked"]:
        x[rand(B, V) < c["masked"]] = -math.inf
        x[:, 0] = 0.0
    s["x"] = x.to(DTYPES[c["x"]])
    s["u"] = torch.rand(B, generator=g, device=dev, dtype=torch.float64)

    def each(v, others, dtype):
        t = torch.full((B,), v, device=dev, dtype=dtype)
        if c["mixed"]:   # a request's own setting
            pick = torch.randint(0, len(others), (B,), generator=g, device=dev)
            t = torch.tensor(others, device=dev, dtype=dtype)[pick]
        return t

    s["temp"] = each(c["temp"], [c["temp"], c["temp"], 0.0, 0.7, 1.2], torch.float32)
    s["k"] = each(c["k"], [c["k"], 0, 20, 200, V // 2], torch.int32)
    s["p"] = each(c["p"], [c["p"], 1.0, 0.9, 0.98], torch.float32)
    s["min_p"] = each(c["min_p"], [c["min_p"], 0.0, 0.02], torch.float32)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _plain_kv(c, s):
    """Ended requests (fresh < 0) push their pages on the stack of free pages; the others take the
    pages they lack from its top, in the order of requests; a request is left out if the table's
    row, the pages left (counting what all before it wanted) or the T token rows do not suffice."""
    page, per, T = c["page"], c["per"], c["T"]
    cached, fresh, blocks, free = s["cached"].long(), s["fresh"].long(), s["blocks"], s["free"]
    F, B = free.numel(), c["B"]
    dev = cached.device
    col = torch.arange(per, device=dev)
    have = (cached + page - 1) // page
    ended = fresh < 0
    # pages of ended requests
    back = torch.where(ended, have, 0)
    at = s["count"].long() + (back.cumsum(0) - back)[:, None] + col
    at = torch.where(ended[:, None] & (col < have[:, None]), at, F)
    stack = torch.cat((free, free[:1]))
    stack[at] = blocks
    free.copy_(stack[:F])
    count = s["count"].long() + back.sum()
    # who is served
    want = torch.where(ended, 0, fresh)
    need = (cached + want + page - 1) // page
    extra = torch.where(ended, 0, need - have)
    served = ~ended & (need <= per) & ((extra == 0) | (extra.cumsum(0) <= count)) & (want.cumsum(0) <= T)
    extra, want = torch.where(served, extra, 0), torch.where(served, want, 0)
    lens = torch.where(ended, 0, cached + want)
    # their new pages
    first = extra.cumsum(0) - extra
    take = count - 1 - (first[:, None] + col - have[:, None])
    fill = (col >= have[:, None]) & (col < (have + extra)[:, None])
    blocks.copy_(torch.where(fill, free[take.clamp(0, F - 1)], blocks))
    # rows of the tokens
    starts = torch.cat((want.new_zeros(1), want.cumsum(0)))
    t = torch.arange(T, device=dev)
    live = t < starts[-1]
    seq = torch.searchsorted(starts, t, right=True) - 1
    seq = torch.where(live, seq, 0).clamp(max=B - 1)
    pos = torch.where(live, cached[seq] + t - starts[seq], 0)
    slot = blocks[seq, pos // page].long() * page + pos % page
    return {"seq": torch.where(live, seq, -1).int(), "pos": torch.where(live, pos, -1).int(),
            "slot": torch.where(live, slot, -1), "lens": lens.int(), "starts": starts.int(),
            "count": (count - extra.sum()).int().view(1), "blocks": blocks, "free": free}


def _plain_embed(c, s):
    ids = s["ids"].long()
    y = s["table"][ids.clamp(min=0)].float() * s["scale"]
    return {"y": torch.where(ids[:, None] >= 0, y, 0.0).to(DTYPES[c["y"]])}


def _plain_embed_bwd(c, s):
    ids = s["ids"].long()
    d = torch.where(ids[:, None] >= 0, s["dy"].float() * s["scale"], 0.0)
    out = s["dtable"] if c["accum"] else d.new_zeros(c["V"], c["K"])
    return {"dtable": out.index_add_(0, ids.clamp(min=0), d)}


def _plain_q4(c, s):
    n, K, group = c["n"], c["K"], c["group"]
    w = (s["q"].float().view(n, K // group, group) * s["scales"].float()[..., None]).view(n, K)
    return {"y": torch.matmul(s["xq"].float(), w.t()) * s["scale"][:, None]}


def _plain_sample(c, s):
    B, V = c["B"], c["V"]
    x, order = s["x"].float().sort(dim=-1, descending=True, stable=True)
    x = x.double()
    top = x[:, :1]
    temp, k, p, min_p, u = (s[n].double()[:, None] for n in ("temp", "k", "p", "min_p", "u"))
    one = torch.full_like(top, 2.0 ** 40)
    # weights are whole numbers: sums of them are exact in any order
    w = torch.exp((x - top) / torch.where(temp > 0, temp, 1.0)) * one
    w = w.round().long()
    rank = torch.arange(V, device=x.device)
    w = torch.where((k <= 0) | (rank < k), w, 0)                                     # top-k
    before = w.cumsum(-1) - w
    goal = p * w.sum(-1, keepdim=True).double()
    keep = (rank == 0) | (((p >= 1) | (before.double() < goal)) & (w.double() >= min_p * one))
    keep = keep & ((temp > 0) | (rank == 0))                                         # greedy
    total = (w * keep).sum(-1, keepdim=True)
    r = torch.minimum((u * total.double()).long(), total - 1)
    n = ((w * keep).cumsum(-1) <= r).sum(-1, keepdim=True).clamp(max=V - 1)
    token = order.gather(-1, n)
    lse = torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    logprob = (x.gather(-1, n) - top - lse).float()
    return {"token": token.int().view(B), "logprob": logprob.view(B)}


PLAIN = {"kv": _plain_kv, "embed": _plain_embed, "embed_bwd": _plain_embed_bwd, "q4": _plain_q4,
         "sample": _plain_sample}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return PLAIN[op](c, s)
    L = _lib()
    if op == "kv":
        r = L.kv_step(s["cached"], s["fresh"], s["blocks"], s["free"], s["count"], c["page"], c["T"])
        return {"seq": r.seq, "pos": r.pos, "slot": r.slot, "lens": r.lens, "starts": r.starts,
                "count": r.count, "blocks": s["blocks"], "free": s["free"]}
    if op == "embed":
        return {"y": L.embed(s["ids"], s["table"], scale=s["scale"], dtype=DTYPES[c["y"]])}
    if op == "embed_bwd":
        return {"dtable": L.embed_bwd(s["dy"], s["ids"], c["V"], scale=s["scale"],
                                      accumulate=c["accum"], out=s.get("dtable"))}
    if op == "q4":
        return {"y": L.q4_fwd(s["xq"], s["scale"], c["K"], s["codes"], s["scales"], c["n"],
                              group=c["group"])}
    token, logprob = L.sample(s["x"], s["u"], temperature=s["temp"], top_k=s["k"], top_p=s["p"],
                              min_p=s["min_p"], want_logprob=True)
    return {"token": token, "logprob": logprob}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_token(x, u, temp, k, p, min_p):
    """One row's token, walking down its values: how many of them stay, then where u falls."""
    order = np.lexsort((np.arange(len(x)), -x))
    if temp <= 0:
        return order[0]
    if 0 < k < len(order):
        order = order[:k]
    w = np.rint(np.exp((x[order] - x[order[0]]) / temp) * 2.0 ** 40).astype(np.int64)
    sums = np.cumsum(w)
    keep = len(w)
    if p < 1:
        keep = 1 + int(np.searchsorted(sums, math.ceil(p * float(sums[-1]))))
    keep = min(keep, max(1, int((w >= min_p * 2.0 ** 40).sum())), len(w))
    r = min(int(u * float(sums[keep - 1])), int(sums[keep - 1]) - 1)
    return order[int(np.searchsorted(sums[:keep], r, side="right"))]


def exact(c, seed):
    op = c["op"]
    if op == "kv":   # whole numbers alone
        return None
    s = prepare(c, seed)
    if op == "embed":
        ids = s["ids"].long()
        y = torch.zeros(c["T"], c["K"], dtype=torch.float64, device=ids.device)
        y[ids >= 0] = s["table"][ids[ids >= 0]].double() * s["scale"]
        return {"y": y}
    if op == "embed_bwd":
        live = torch.nonzero(s["ids"] >= 0)[:, 0]
        ids, order = s["ids"][live].long().sort(stable=True)
        out = torch.zeros(c["V"], c["K"], dtype=torch.float64, device=ids.device)
        if c["accum"]:
            out += s["dtable"]
        for i in range(0, len(live), 4096):   # runs of equal ids by sums up to their ends
            at, d = ids[i:i + 4096], s["dy"][live[order[i:i + 4096]]].double().cumsum(0)
            last = torch.ones_like(at, dtype=torch.bool)
            last[:-1] = at[1:] != at[:-1]
            end = d[last]
            end[1:] -= d[last][:-1]
            out[at[last]] += end * s["scale"]
        return {"dtable": out}
    if op == "q4":
        n, K, group = c["n"], c["K"], c["group"]
        if own:
            return None
        y = torch.empty(c["T"], n, dtype=torch.float64, device=s["xq"].device)
        x = s["xq"].double().view(c["T"], K // group, group)
        for i in range(0, n, 8192):   # a group's sum first, then its scale
            q = s["q"][i:i + 8192].double().view(-1, K // group, group)
            dots = torch.matmul(x.transpose(0, 1).contiguous(), q.permute(1, 2, 0).contiguous())
            y[:, i:i + 8192] = (dots * s["scales"][i:i + 8192].double().t()[:, None]).sum(0)
        return {"y": y * s["scale"].double()[:, None]}
    x = s["x"].double().cpu()
    token = torch.tensor([int(_exact_token(x[b].numpy(), *(s[n][b].item() for n in ("u", "temp", "k", "p", "min_p"))))
                          for b in range(c["B"])])
    return {"token": None, "logprob": torch.log_softmax(x, -1)[torch.arange(c["B"]), token]}
