"""What is measured of the 8-bit operators: the block-scaled e4m3 product with its quantizer, and the
e4m3 KV cache with its append, attention and eviction.

Blocks carry power-of-two scales: s is the smallest 2^e in 2^-40 .. 2^40 with amax <= 448 s, and a
value x is held as the e4m3 number nearest to x / s (ties to even).

  quantize  x[R, C] -> codes and a scale for each 1 x 128 (activations) or 128 x 128 (weights) block
  gemm      Y[m, n] = sum_t sa[t, m] sw[t, n / 128] sum_{k in block t} A[m, k] W[n, k]
  append    writes new tokens behind each sequence of a paged cache [page][head][token][dim] that has
            one scale per page and head; a page's scale grows with its tokens, its older codes follow
  attend    softmax(scale q k^T) v over each sequence's pages, queries at the end of the sequence;
            also the log of the sums and, if asked, the weights each cached token received
  evict     keeps the last tokens and the best of the others by accumulated weight, in order, and
            moves them to other pages

Sizes: 32 heads of 128, sequences of 8192 and batch 8 are the KV workload of this repository's
benchmark, 4096 x 4096 and 11008 x 4096 its weight workload.
"""
import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decoding step's activations before a projection: latency
        {"name": "quantize-step", "op": "quantize", "rows": 8, "cols": 4096, "block": 1, "dtype": "bf16"},
        # one MLP weight brought into 8 bits when a model is loaded
        {"name": "quantize-weight", "op": "quantize", "rows": 11008, "cols": 4096, "block": 128, "dtype": "bf16"},
        # a decoding step's attention projection: the weight's bytes count
        {"name": "gemm-step", "op": "gemm", "m": 7, "n": 4096, "k": 4096, "dtype": "bf16"},
        # a short prompt through odd sizes with a binary32 result (logits)
        {"name": "gemm-ragged", "op": "gemm", "m": 333, "n": 1000, "k": 1460, "dtype": "f32"},
        # a long prompt through the MLP projection
        {"name": "gemm-prompt", "op": "gemm", "m": 4096, "n": 11008, "k": 4096, "dtype": "bf16"},
        # one new token of eight sequences
        {"name": "append-step", "op": "append", "batch": 8, "heads": 32, "dim": 128, "page": 64, "new": 1,
         "most": 2000, "ragged": False, "dtype": "bf16"},
        # prompts of unequal length, padded, behind what the cache holds
        {"name": "append-prompt", "op": "append", "batch": 8, "heads": 32, "dim": 128, "page": 64, "new": 2048,
         "most": 700, "ragged": True, "dtype": "bf16"},
        # a decoding step over the benchmark's KV cache
        {"name": "attend-step", "op": "attend", "batch": 8, "heads": 32, "group": 1, "dim": 128, "page": 64, "queries": 1,
         "length": 8192, "ragged": False, "weights": False},
        # a few speculative tokens, grouped heads of 64, short ragged sequences, small pages, weights for eviction
        {"name": "attend-few", "op": "attend", "batch": 3, "heads": 8, "group": 5, "dim": 64, "page": 16, "queries": 2,
         "length": 1500, "ragged": True, "weights": True},
        # a chunk of a long prompt behind its cached beginning
        {"name": "attend-chunk", "op": "attend", "batch": 2, "heads": 8, "group": 4, "dim": 128, "page": 64, "queries": 512,
         "length": 8192, "ragged": False, "weights": False},
        # a small cache brought down to its budget between two steps
        {"name": "evict-small", "op": "evict", "batch": 1, "heads": 8, "dim": 64, "page": 16, "length": 1100, "budget": 500,
         "recent": 33, "ragged": False},
        # the benchmark's KV cache brought down to a quarter
        {"name": "evict-long", "op": "evict", "batch": 8, "heads": 32, "dim": 128, "page": 64, "length": 8192,
         "budget": 2048, "recent": 256, "ragged": False},
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "append", "attend", "attend", "evict"])
    if op == "quantize":
        cols = _log(rng, 1, 8192)
        return {"op": op, "rows": _log(rng, 1, min(11008, 45000000 // cols)), "cols": cols, "block": rng.choice([1, 128]),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "gemm":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 1, 11008), "k": _log(rng, 1, 4096),
                "dtype": rng.choice(["bf16", "f32"])}
    heads, dim, page = rng.choice([1, 2, 4, 8, 10, 32]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        new = _log(rng, 1, 2048)
        return {"op": op, "batch": _log(rng, 1, max(1, min(64, 8 * 2048 // new))), "heads": heads, "dim": dim, "page": page,
                "new": new, "most": _log(rng, 1, 2000), "ragged": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f32"])}
    if op == "attend":
        length = _log(rng, 1, 8192)
        queries = 1 if rng.random() < 0.4 else _log(rng, 1, min(512, length + 2))
        group = rng.choice([1, 2, 3, 4, 5, 8])
        batch = _log(rng, 1, 64)
        batch = max(1, min(batch, 8 * 32 * 8192 // (length * heads), 2 * 32 * 512 * 8192 // (heads * group * queries * length)))
        return {"op": op, "batch": batch, "heads": heads, "group": group, "dim": dim, "page": page, "queries": queries,
                "length": length, "ragged": rng.random() < 0.6, "weights": rng.random() < 0.4}
    length = _log(rng, 2, 8192)
    return {"op": op, "batch": max(1, min(_log(rng, 1, 16), 8 * 32 * 8192 // (length * heads))), "heads": heads, "dim": dim,
            "page": page, "length": length, "budget": _log(rng, 1, length), "recent": _log(rng, 1, 512) - 1,
            "ragged": rng.random() < 0.5}


def _ceil(a, b):
    return -(-a // b)


def work(c):
    op = c["op"]
    if op == "quantize":
        n, t = c["rows"] * c["cols"], _ceil(c["cols"], 128) * _ceil(c["rows"], c["block"])
        return {"bytes": n * (3 if c["dtype"] == "bf16" else 5) + 4 * t, "flops": 3 * n}
    if op == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * k + m * n * (2 if c["dtype"] == "bf16" else 4) + 4 * _ceil(k, 128) * (m + _ceil(n, 128)),
                "flops": 2 * m * n * k}
    if op == "append":
        n = 2 * c["batch"] * c["heads"] * c["dim"] * (c["new"] * (0.5 if c["ragged"] and c["new"] > 1 else 1))
        return {"bytes": n * (3 if c["dtype"] == "bf16" else 5), "flops": 3 * n}
    if op == "attend":
        tokens = c["batch"] * c["heads"] * c["length"] * (0.5 if c["ragged"] else 1.0)
        rows = c["group"] * c["queries"]
        qo = 4 * c["batch"] * c["heads"] * rows * c["dim"]
        return {"bytes": tokens * (2 * c["dim"] + (8 if c["weights"] else 0)) + qo, "flops": 4 * tokens * rows * c["dim"]}
    tokens = c["batch"] * c["heads"]
    return {"bytes": tokens * (4 * c["length"] + min(c["budget"], c["length"]) * (4 * c["dim"] + 4)), "flops": tokens * c["length"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _fit(amax):
    """The scale of a block whose largest magnitude is `amax` (binary32)."""
    mant, ex = torch.frexp(amax)  # amax = mant 2^ex, mant in [1/2, 1); 448 = 0.875 2^9
    e = torch.where(mant > 0.875, ex - 8, ex - 9).clamp(-40, 40)
    e = torch.where(amax > 0, e, torch.full_like(e, -40))
    return torch.ldexp(torch.ones_like(amax), e)


def _cache(g, pool, heads, page, dim):
    """A filled pool: keys with four strong channels per head, values without; pages of unlike loudness."""
    loud = torch.exp(0.4 * torch.randn(pool, 1, 1, 1, device="cuda", generator=g))
    strong = torch.ones(1, heads, 1, dim, device="cuda")
    strong.scatter_(3, torch.rand(1, heads, 1, dim, device="cuda", generator=g).topk(4, dim=3).indices, 10.0)
    k = torch.randn(pool, heads, page, dim, device="cuda", generator=g) * strong
    ks = _fit(k.abs().amax((2, 3)))
    k = (k / ks[:, :, None, None]).to(F8)
    v = torch.randn(pool, heads, page, dim, device="cuda", generator=g) * loud
    vs = _fit(v.abs().amax((2, 3)))
    return k, (v / vs[:, :, None, None]).to(F8), ks, vs


def _lens(c, g, most):
    """int32 [batch]: all `most`, or ragged 0 .. most with the longest among them."""
    if not c["ragged"]:
        return torch.full((c["batch"],), most, dtype=torch.int32, device="cuda")
    lens = torch.randint(0, most + 1, (c["batch"],), device="cuda", generator=g, dtype=torch.int32)
    lens[0] = most
    return lens


def _table(g, batch, pages, spare):
    """Pages of every sequence, in no order, and the pool's size."""
    pool = batch * pages + spare
    return torch.randperm(pool, device="cuda", generator=g)[:batch * pages].view(batch, pages).to(torch.int32), pool


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = c["op"]
    if op == "quantize":
        x = torch.randn(c["rows"], c["cols"], device="cuda", generator=g)
        x *= torch.exp(torch.randn(1, c["cols"], device="cuda", generator=g))  # channels of unlike size
        x[:, c["cols"] // 2:c["cols"] // 2 + 1] *= 20.0
        x[c["rows"] // 2, :130] = 0.0  # blocks of zeros
        return {"c": c, "x": (0.02 * x).to(DTYPES[c["dtype"]])}
    if op == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        kb, ld = _ceil(k, 128), _ceil(k, 16) * 16
        a = torch.zeros(m, ld, device="cuda")
        a[:, :k] = 100.0 * torch.randn(m, k, device="cuda", generator=g)
        w = torch.zeros(n, ld, device="cuda")
        w[:, :k] = 100.0 * torch.randn(n, k, device="cuda", generator=g)
        sa = torch.exp2(torch.randint(-8, -3, (kb, m), device="cuda", generator=g).float())
        sw = torch.exp2(torch.randint(-14, -11, (kb, _ceil(n, 128)), device="cuda", generator=g).float())
        return {"c": c, "a": a.clamp(-448, 448).to(F8), "sa": sa, "w": w.clamp(-448, 448).to(F8), "sw": sw}
    b, h, d, page = c["batch"], c["heads"], c["dim"], c["page"]
    if op == "append":
        table, pool = _table(g, b, _ceil(c["most"] + c["new"], page), 3)
        k, v, ks, vs = _cache(g, pool, h, page, d)
        dt = DTYPES[c["dtype"]]
        # one projection's rows [batch, token, k heads | v heads, dim]: the views are strided
        kv = torch.randn(b, c["new"], 2 * h, d, device="cuda", generator=g).to(dt)
        lens = torch.randint(0, c["most"] + 1, (b,), device="cuda", generator=g, dtype=torch.int32)
        new = _lens(c, g, c["new"])
        return {"c": c, "k": k, "v": v, "ks": ks, "vs": vs, "table": table, "lens": lens, "new": new,
                "xk": kv[:, :, :h].transpose(1, 2), "xv": kv[:, :, h:].transpose(1, 2)}
    if op == "attend":
        length, sq, hq = c["length"], c["queries"], c["heads"] * c["group"]
        table, pool = _table(g, b, _ceil(length, page), 2)
        k, v, ks, vs = _cache(g, pool, h, page, d)
        q = torch.randn(b, sq, hq, d, device="cuda", generator=g).to(torch.bfloat16).transpose(1, 2)
        s = {"c": c, "k": k, "v": v, "ks": ks, "vs": vs, "table": table, "lens": _lens(c, g, length), "q": q,
             "qlens": _lens(c, g, sq), "out": torch.zeros(b, hq, sq, d, device="cuda", dtype=torch.bfloat16),
             "lse": torch.zeros(b, hq, sq, device="cuda")}
        if c["weights"]:
            s["win"] = torch.rand(b, h, length, device="cuda", generator=g)
            s["wout"] = torch.zeros(b, h, length, device="cuda")
        return s
    length, keep = c["length"], min(c["budget"], c["length"])
    tables, pool = _table(g, b, _ceil(length, page) + _ceil(keep, page), 2)
    k, v, ks, vs = _cache(g, pool, h, page, d)
    w = torch.exp(3.0 * torch.randn(b, h, length, device="cuda", generator=g))
    w = torch.where(torch.rand(b, h, length, device="cuda", generator=g) < 0.1, torch.zeros_like(w), w)  # ties
    return {"c": c, "k": k, "v": v, "ks": ks, "vs": vs, "table": tables[:, :_ceil(length, page)].contiguous(),
            "to": tables[:, _ceil(length, page):].contiguous(), "lens": _lens(c, g, length), "w": w,
            "olens": torch.zeros(b, dtype=torch.int32, device="cuda"), "ow": torch.zeros(b, h, keep, device="cuda")}


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    return {"quantize": _quantize, "gemm": _gemm, "append": _append, "attend": _attend, "evict": _evict}[s["c"]["op"]](s)


def _quantize(s):
    x, block = s["x"], s["c"]["block"]
    if own:
        import post_quantization_tile_b200 as hq
        code = hq.fp8_quantize(x, block=block)
        return code.data, code.scale
    rows, cols = x.shape
    ld, kb, rb = _ceil(cols, 16) * 16, _ceil(cols, 128), _ceil(rows, block)
    y = torch.zeros(rb * block, kb * 128, device=x.device)
    y[:rows, :cols] = x
    y = y.view(rb, block, kb, 128)
    scale = _fit(y.abs().amax((1, 3)))
    q = (y / scale[:, None, :, None]).clamp(-448, 448).to(F8)
    return q.view(rb * block, kb * 128)[:rows, :ld].contiguous(), scale.t().contiguous()


def _gemm(s):
    c, dt = s["c"], DTYPES[s["c"]["dtype"]]
    if own:
        import post_quantization_tile_b200 as hq
        a = hq.Fp8Code(c["m"], c["k"], 1, s["a"], s["sa"])
        return hq.gemm_fp8(a, hq.Fp8Code(c["n"], c["k"], 128, s["w"], s["sw"]), dtype=dt)
    a = s["a"].float() * s["sa"].t().repeat_interleave(128, 1)[:, :s["a"].shape[1]]
    w = s["w"].float() * s["sw"].t().repeat_interleave(128, 1)[:, :s["w"].shape[1]].repeat_interleave(128, 0)[:c["n"]]
    return (a @ w.t()).to(dt)


def _append_one(codes, scale, x, table, lens, new):
    b, h, n, d = x.shape
    page = codes.shape[2]
    span = min(_ceil(n, page) + 1, table.shape[1])  # pages that the new tokens can touch
    at = lens[:, None].long() // page + torch.arange(span, device=x.device)
    slot = at[:, :, None] * page + torch.arange(page, device=x.device)  # [b, span, page]
    t = slot - lens[:, None, None]
    fresh = (t >= 0) & (t < new[:, None, None])
    old = t < 0
    ids = table.gather(1, at.clamp(max=table.shape[1] - 1)).long()
    took = x.float().gather(2, t.clamp(0, n - 1).view(b, 1, -1, 1).expand(b, h, -1, d))
    took = took.view(b, h, span, page, d).transpose(1, 2)  # [b, span, h, page, d]
    f = fresh[:, :, None, :, None]
    s_new = _fit(torch.where(f, took.abs(), torch.zeros_like(took)).amax((3, 4)))
    s_old = scale[ids]
    s = torch.where(old.any(2)[:, :, None], torch.maximum(s_old, s_new), s_new)
    had = codes.view(torch.uint8)[ids].view(F8).float()
    s_ = s[:, :, :, None, None]
    q = torch.where(f, took / s_, torch.where(old[:, :, None, :, None], had * (s_old[:, :, :, None, None] / s_), had))
    touched = fresh.any(2)
    codes.view(torch.uint8)[ids[touched]] = q.to(F8).view(torch.uint8)[touched]
    scale[ids[touched]] = s[touched]


def _append(s):
    if own:
        import post_quantization_tile_b200 as hq
        hq.kv8_append(hq.Kv8Cache(s["k"], s["v"], s["ks"], s["vs"]), s["xk"], s["xv"], s["table"], s["lens"], n_new=s["new"])
    else:
        _append_one(s["k"], s["ks"], s["xk"], s["table"], s["lens"], s["new"])
        _append_one(s["v"], s["vs"], s["xv"], s["table"], s["lens"], s["new"])
    return s["k"], s["v"], s["ks"], s["vs"]


def _gathered(codes, scale, table):
    """The cache of each sequence as binary32 values [batch, heads, slots, dim]."""
    ids = table.long()
    x = codes.view(torch.uint8)[ids].view(F8).float() * scale[ids][:, :, :, None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend(s):
    c = s["c"]
    if own:
        import post_quantization_tile_b200 as hq
        hq.kv8_attend(s["q"], hq.Kv8Cache(s["k"], s["v"], s["ks"], s["vs"]), s["table"], s["lens"], q_lens=s["qlens"],
                      out=s["out"], lse=s["lse"], weights=s.get("wout"), weights_in=s.get("win"))
        return [s["out"], s["lse"]] + ([s["wout"]] if c["weights"] else [])
    b, h, group, sq, d, length = c["batch"], c["heads"], c["group"], c["queries"], c["dim"], c["length"]
    k, v = _gathered(s["k"], s["ks"], s["table"])[:, :, :length], _gathered(s["v"], s["vs"], s["table"])[:, :, :length]
    q = s["q"].float().reshape(b, h, group * sq, d)
    i, j = torch.arange(sq, device="cuda"), torch.arange(length, device="cuda")
    lens, ql = s["lens"][:, None, None].long(), s["qlens"][:, None, None].long()
    asked = i[None, :, None] < ql
    sees = (j[None, None, :] < lens - ql + i[None, :, None] + 1) & asked  # [b, sq, length]
    x = (q @ k.transpose(2, 3)).view(b, h, group, sq, length) * (d ** -0.5)
    x = torch.where(sees[:, None, None], x, torch.full_like(x, -torch.inf))
    top = x.amax(4, keepdim=True)
    p = torch.exp(x - torch.where(top > -torch.inf, top, torch.zeros_like(top)))
    total = p.sum(4, keepdim=True)
    some = torch.where(total > 0, total, torch.ones_like(total))
    o = ((p.view(b, h, group * sq, length) @ v).view(b, h, group, sq, d) / some).reshape(b, h * group, sq, d)
    rows = asked.view(b, 1, sq)
    s["out"].copy_(torch.where(rows[..., None], o.to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(rows, (top + torch.log(total)).view(b, h * group, sq), s["lse"]))
    if not c["weights"]:
        return [s["out"], s["lse"]]
    w = s["win"] + (p / some).sum((2, 3))
    s["wout"].copy_(torch.where(j < lens, w, s["wout"]))
    return [s["out"], s["lse"], s["wout"]]


def _evict(s):
    c = s["c"]
    keep = min(c["budget"], c["length"])
    if own:
        import post_quantization_tile_b200 as hq
        hq.kv8_evict(hq.Kv8Cache(s["k"], s["v"], s["ks"], s["vs"]), s["table"], s["lens"], s["w"], keep, c["recent"], s["to"],
                     out_lens=s["olens"], out_weights=s["ow"])
        return s["k"], s["v"], s["ks"], s["vs"], s["olens"], s["ow"]
    b, h, page, length = c["batch"], c["heads"], c["page"], c["length"]
    lens = s["lens"][:, None, None].long()
    j = torch.arange(length, device="cuda")
    recent = min(c["recent"], keep)
    # recent tokens first, then by weight, lowest index first among equals; slots past the end last
    rank = torch.where(j >= lens - recent, torch.full_like(s["w"], torch.inf), s["w"])
    rank = torch.where(j < lens, rank, torch.full_like(rank, -torch.inf))
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :keep]
    n = torch.minimum(s["lens"], torch.full_like(s["lens"], keep))
    i = torch.arange(keep, device="cuda")
    valid = (i < n[:, None, None].long()).expand(b, h, keep)
    src = torch.sort(torch.where(valid, order, torch.full_like(order, length)), dim=2).values.clamp(max=length - 1)
    _move(s["k"], s["ks"], s["table"], s["to"], src, valid)
    _move(s["v"], s["vs"], s["table"], s["to"], src, valid)
    s["ow"].copy_(torch.where(valid, s["w"].gather(2, src), s["ow"]))
    s["olens"].copy_(n)
    return s["k"], s["v"], s["ks"], s["vs"], s["olens"], s["ow"]


def _move(codes, scale, table, to, src, valid):
    b, h, keep = src.shape
    page = codes.shape[2]
    heads = torch.arange(h, device="cuda")[None, :, None]
    ids = table.long().gather(1, (src // page).view(b, -1)).view(b, h, keep)
    had = codes.view(torch.uint8)[ids, heads, src % page].view(F8).float()
    s_had = torch.where(valid, scale[ids, heads], torch.zeros_like(scale[ids, heads]))
    pages = to.shape[1]
    pad = torch.zeros(b, h, pages * page - keep, device="cuda")
    s_to = torch.cat([s_had, pad], 2).view(b, h, pages, page).amax(3)
    i = torch.arange(keep, device="cuda")
    q = (had * (s_had / s_to[:, :, i // page])[..., None]).to(F8).view(torch.uint8)
    at = to.long()[:, i // page][:, None].expand(b, h, keep)
    codes.view(torch.uint8)[at[valid], heads.expand(b, h, keep)[valid], (i % page).expand(b, h, keep)[valid]] = q[valid]
    some = s_to > 0
    at = to.long()[:, None].expand(b, h, pages)
    scale[at[some], heads.expand(b, h, pages)[some]] = s_to[some]


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _np(t):
    return t.detach().cpu().double().numpy()


def _scale_of(amax):
    """2^ceil(log2(amax / 448)) by whole-number search, in 2^-40 .. 2^40."""
    e = np.clip(np.floor(np.log2(np.maximum(amax, 1e-300) / 448.0)).astype(np.int64) - 1, -40, 40)
    for _ in range(3):
        e = np.where((448.0 * 2.0 ** e < amax) & (e < 40), e + 1, e)
    return 2.0 ** e


def _nearest(y):
    """The e4m3 number nearest to y, ties to the even code."""
    step = 2.0 ** np.clip(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -30))), -6, None) / 8.0
    return np.clip(np.rint(y / step) * step, -448.0, 448.0)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "quantize":
        x = _np(s["x"])
        q = np.zeros((c["rows"], _ceil(c["cols"], 16) * 16))
        scale = np.zeros((_ceil(c["cols"], 128), _ceil(c["rows"], c["block"])))
        for t in range(scale.shape[0]):
            at = x[:, 128 * t:128 * t + 128]
            scale[t] = _scale_of(np.maximum.reduceat(np.abs(at).max(1), np.arange(0, c["rows"], c["block"])))
            q[:, 128 * t:128 * t + at.shape[1]] = _nearest(at / np.repeat(scale[t], c["block"])[:c["rows"], None])
        return q, scale
    if op == "gemm":
        y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
        for t in range(s["sa"].shape[0]):
            part = s["a"][:, 128 * t:128 * t + 128].double() @ s["w"][:, 128 * t:128 * t + 128].double().t()
            y += part * s["sa"][t].double()[:, None] * torch.repeat_interleave(s["sw"][t].double(), 128)[:c["n"]]
        return y
    table, lens, page = _np(s["table"]).astype(np.int64), _np(s["lens"]).astype(np.int64), c["page"]
    if op == "append":
        new, outs = _np(s["new"]).astype(np.int64), []
        if s["k"].numel() > 1 << 28:
            return None
        for codes, scale, x in ((s["k"], s["ks"], s["xk"]), (s["v"], s["vs"], s["xv"])):
            codes, scale, x = _np(codes), _np(scale), _np(x)
            for b in range(c["batch"]):
                first, last = lens[b], lens[b] + new[b]
                for p in range(first // page, _ceil(last, page) if new[b] else 0):
                    lo, hi = max(first, p * page), min(last, (p + 1) * page)
                    at, held = table[b, p], lo - p * page
                    take = x[b, :, lo - first:hi - first]
                    to = _scale_of(np.abs(take).max((1, 2)))
                    if held:
                        to = np.maximum(to, scale[at])
                        codes[at, :, :held] = _nearest(codes[at, :, :held] * (scale[at] / to)[:, None, None])
                    codes[at, :, held:hi - p * page] = _nearest(take / to[:, None, None])
                    scale[at] = to
            outs.append((codes, scale))
        return outs[0][0], outs[1][0], outs[0][1], outs[1][1]
    if op == "attend":
        qlens = _np(s["qlens"]).astype(np.int64)
        out, lse = s["out"].double(), s["lse"].double()
        w = s["wout"].double() if c["weights"] else None
        for b in range(c["batch"]):
            n, m = int(lens[b]), int(qlens[b])
            ids = s["table"][b, :_ceil(n, page)].long()
            for h in range(c["heads"]):
                k = (s["k"][ids, h].double() * s["ks"][ids, h].double()[:, None, None]).reshape(-1, c["dim"])[:n]
                v = (s["v"][ids, h].double() * s["vs"][ids, h].double()[:, None, None]).reshape(-1, c["dim"])[:n]
                heads = slice(h * c["group"], (h + 1) * c["group"])
                x = s["q"][b, heads, :m].double() @ k.t() / math.sqrt(c["dim"])
                behind = torch.arange(n, device="cuda") > torch.arange(m, device="cuda")[:, None] + (n - m)
                x = x.masked_fill(behind, -math.inf)
                p = torch.nan_to_num(torch.softmax(x, 2))
                out[b, heads, :m] = p @ v
                lse[b, heads, :m] = torch.logsumexp(x, 2) if n else -math.inf
                if w is not None:
                    w[b, h, :n] = s["win"][b, h, :n].double() + p.sum((0, 1))
        return [out, lse] + ([w] if w is not None else [])
    keep = min(c["budget"], c["length"])
    k, v, ks, vs = _np(s["k"]), _np(s["v"]), _np(s["ks"]), _np(s["vs"])
    w, to, ow, olens = _np(s["w"]), _np(s["to"]).astype(np.int64), _np(s["ow"]), np.minimum(lens, keep)
    for b in range(c["batch"]):
        n, last = int(lens[b]), int(min(c["recent"], keep, lens[b]))
        for h in range(c["heads"]):
            kept = np.arange(n)
            if n > keep:
                best = np.lexsort((np.arange(n - last), -w[b, h, :n - last]))[:keep - last]
                kept = np.sort(np.concatenate([best, np.arange(n - last, n)]))
            ow[b, h, :kept.size] = w[b, h, kept]
            at = table[b, kept // page]
            for codes, scale in ((k, ks), (v, vs)):
                had, s_had = codes[at, h, kept % page], scale[at, h]
                for p in range(_ceil(kept.size, page)):
                    part = slice(p * page, min((p + 1) * page, kept.size))
                    top = s_had[part].max()
                    codes[to[b, p], h, :part.stop - part.start] = _nearest(had[part] * (s_had[part] / top)[:, None])
                    scale[to[b, p], h] = top
    return k, v, ks, vs, olens, ow
