"""Measured cases of the operators that serve a prompt and its continuation with an 8-bit paged K/V cache.

Three operators, each in its plain form (torch, 32 bits) and, with ``own``, as
the calls a user makes of this framework:

  append  the projections' queries and keys rotated by their positions, the
          keys and values quantized to e4m3 and appended to the paged cache,
          with a power-of-two scale for each page, side and head that grows
          with what the page holds;
  paged   attention that reads that cache: causal, with a sliding window and a
          few first tokens that stay visible, for single decoded tokens and
          for chunks of new tokens;
  prompt  attention over whole prompts before anything of them is quantized:
          causal, grouped heads, packed sequences of different lengths.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
LEAST, MOST = -60, 60                                    # exponents that a page's scale can have
BIAS = 127                                               # a scale byte holds exponent + BIAS


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _append(name, batch, new, ctx_lo, ctx_hi, heads, kv_heads, dim, page, layout, rot, interleaved=False, ragged=False):
    return {"name": name, "op": "append", "batch": batch, "new": new, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "layout": layout, "rot": rot,
            "interleaved": interleaved, "ragged": ragged}


def _paged(name, batch, new, ctx_lo, ctx_hi, heads, kv_heads, dim, page, layout, window=0, sinks=0, ragged=False):
    return {"name": name, "op": "paged", "batch": batch, "new": new, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "layout": layout, "window": window,
            "sinks": sinks, "ragged": ragged}


def _prompt(name, batch, new, heads, kv_heads, dim, window=0, sinks=0, ragged=False):
    return {"name": name, "op": "prompt", "batch": batch, "new": new, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "window": window, "sinks": sinks, "ragged": ragged}


def listed():
    return [
        # one user's decode step: latency
        _append("append decode 1", 1, 1, 300, 300, 32, 8, 128, 64, "NHD", 128),
        # a full decode batch: one token in each request's last page
        _append("append decode 128", 128, 1, 40, 400, 32, 8, 128, 16, "NHD", 128),
        # four prompts, or chunks of them: one read and one write of everything
        _append("append prompts 4x4096", 4, 4096, 0, 400, 32, 8, 128, 64, "NHD", 128),
        # odd sizes: 7 query heads per key head, partial rotation of adjacent pairs, pages of 24, head-major cache
        _append("append odd", 9, 500, 0, 300, 21, 3, 64, 24, "HND", 32, True, True),
        # one user's decode step behind a long prompt
        _paged("paged decode 1", 1, 1, 8000, 8000, 32, 8, 128, 64, "NHD"),
        # a full decode batch on a windowed layer
        _paged("paged decode 128", 128, 1, 4096, 16384, 32, 8, 128, 16, "NHD", 4096, 4),
        # a decode batch over the repository's long contexts
        _paged("paged decode 32 full", 32, 1, 7378, 34474, 32, 8, 128, 64, "NHD"),
        # chunks of four long prompts, behind what is cached of them
        _paged("paged chunks 4x2048", 4, 2048, 0, 8192, 32, 8, 128, 64, "NHD"),
        # a batch of short questions
        _prompt("prompt short", 16, 100, 32, 8, 128, ragged=True),
        # odd sizes: 7 query heads per key head of 64, ragged prompts on a windowed layer
        _prompt("prompt odd", 12, 3000, 21, 3, 64, 777, 17, True),
        # four prompts of a full chunk each
        _prompt("prompt 4x4096", 4, 4096, 32, 8, 128),
        # one long document
        _prompt("prompt 1x16384", 1, 16384, 32, 8, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        # no dearer than the largest listed case, in the plain form's memory too
        if w["bytes"] <= 1.3e9 and w["flops"] <= 1.9e12 and _plain_values(c) <= 8e9:
            return c


def _draw(rng):
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8, 8])
    heads = kv * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
    page = rng.choice([16, 16, 24, 32, 64, 64, 128])
    layout = rng.choice(["NHD", "HND"])
    kind = rng.choice(["append", "append", "decode", "decode", "chunk", "chunk", "prompt", "prompt", "prompt"])
    if kind == "append":
        c = _append("", _log(rng, 1, 128), rng.choice([1, _log(rng, 1, 4096)]), 0, _log(rng, 1, 400), heads, kv, dim,
                    page, layout, rng.choice([dim, dim, dim // 2, 32]), rng.random() < 0.3, rng.random() < 0.5)
        if c["batch"] * c["new"] > 16384:
            c["new"] = 16384 // c["batch"]
    elif kind == "prompt":
        c = _prompt("", _log(rng, 1, 64), _log(rng, 1, 12000), heads, kv, dim, rng.choice([0, 0, _log(rng, 16, 4096)]),
                    rng.choice([0, 4, rng.randint(1, 128)]), rng.random() < 0.5)
    else:
        hi = _log(rng, 16, 34000)
        window = rng.choice([0, 0, _log(rng, 1 if kind == "decode" else 16, 8192)])
        sinks = rng.choice([0, 4, rng.randint(1, 128)])
        if kind == "decode":
            c = _paged("", _log(rng, 1, 128), 1, rng.randint(0, hi), hi, heads, kv, dim, page, layout, window, sinks)
        else:
            c = _paged("", _log(rng, 1, 16), _log(rng, 2, 4096), rng.randint(0, hi), hi, heads, kv, dim, page, layout,
                       window, sinks, rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(c):
    """Cached and new tokens of each request: fixed by the case, not by the seed."""
    lo, hi = c.get("ctx_lo", 0), c.get("ctx_hi", 0)
    r = random.Random("%s %s %s %s" % (c["batch"], lo, hi, c["new"]))
    ctx = [r.randint(lo, hi) for _ in range(c["batch"])]
    new = [r.randint(1, c["new"]) if c["ragged"] and b else c["new"] for b in range(c["batch"])]
    return ctx, new


def _visible(c, ctx, new):
    """(keys read at least once, (query, key) pairs) of one request."""
    w, ns = c["window"], c["sinks"]
    total = ctx + new
    if w <= 0:
        return total, new * ctx + new * (new + 1) // 2
    pairs = 0
    for i in range(new):
        p = ctx + i
        lo = max(0, p - w + 1)
        pairs += p + 1 - lo + min(ns, lo)
    first = max(0, ctx - w + 1)
    return total - first + min(ns, first), pairs


def _plain_values(c):
    """Values that the plain form holds at once: scores, or decoded keys."""
    if c["op"] == "append":
        return 0
    keys = c.get("ctx_hi", 0) + c["new"]
    if c["op"] == "paged" and c["window"]:
        keys = min(keys, c["window"] + c["new"]) + c["sinks"]
    return c["batch"] * max(c["heads"] * c["new"] * keys, 2 * c["kv_heads"] * c["dim"] * keys)


def work(c):
    ctx, new = _lengths(c)
    tokens = sum(new)
    if c["op"] == "append":
        # queries and keys read and written, values read, codes written; the table's row and the position of a token
        values = tokens * (4 * c["heads"] + 4 * c["kv_heads"] + 2 * c["kv_heads"] + 2 * c["kv_heads"]) * c["dim"]
        pages = sum((x + n - 1) // c["page"] - x // c["page"] + 1 for x, n in zip(ctx, new))
        return {"bytes": values + tokens * (8 + 4 * c["rot"]) + pages * (2 * c["kv_heads"] + 4),
                "flops": tokens * (4 * (c["heads"] + c["kv_heads"]) * c["rot"] + 4 * c["kv_heads"] * c["dim"])}
    seen = [_visible(c, x, n) for x, n in zip(ctx, new)]
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    flops = 4 * c["dim"] * c["heads"] * pairs
    rows = tokens * c["heads"] * (4 * c["dim"] + 4)
    if c["op"] == "prompt":
        return {"bytes": rows + tokens * c["kv_heads"] * 4 * c["dim"], "flops": flops}
    pages = sum((x + n + c["page"] - 1) // c["page"] for x, n in zip(ctx, new))
    return {"bytes": keys * c["kv_heads"] * 2 * c["dim"] + rows + pages * (4 + 2 * c["kv_heads"]), "flops": flops}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _table(c, totals, gen):
    """Shuffled pages for every request; the columns past a request's last are -1."""
    need = [-(-t // c["page"]) for t in totals]
    pages = sum(need) + 8
    order = torch.randperm(pages, device=DEVICE, generator=gen)[:sum(need)].to(torch.int32).cpu()
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pages, table.to(DEVICE)


def _cache(pages, c, gen):
    """A cache that holds normals: each page, side and head with the scale its
    largest value asks for (2^-7 or 2^-6 for ordinary ones), and codes of a
    normal's quantiles."""
    inner = (c["page"], c["kv_heads"], c["dim"]) if c["layout"] == "NHD" else (c["kv_heads"], c["page"], c["dim"])
    cache = torch.empty((pages, 2, *inner), dtype=torch.uint8, device=DEVICE)
    exponent = torch.randint(-7, -5, (pages, 2, c["kv_heads"]), device=DEVICE, generator=gen)
    x = torch.special.ndtri((torch.arange(256, device=DEVICE, dtype=torch.float64) + 0.5) / 256).float()
    lut = [(x * 2.0 ** -e).to(torch.float8_e4m3fn).view(torch.uint8) for e in (-7, -6)]
    step = max(1, (1 << 28) // (2 * c["page"] * c["kv_heads"] * c["dim"]))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        at = torch.randint(0, 256, (n, 2, *inner), device=DEVICE, generator=gen, dtype=torch.int32)
        e = exponent[i:i + n].view(n, 2, 1, -1, 1) if c["layout"] == "NHD" else exponent[i:i + n].view(n, 2, -1, 1, 1)
        cache[i:i + n] = torch.where(e == -7, lut[0].index_select(0, at.view(-1)).view(at.shape),
                                     lut[1].index_select(0, at.view(-1)).view(at.shape))
    return cache, (exponent + BIAS).to(torch.uint8)


def prepare(c, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(1000 + seed)
    s = {"case": c}
    ctx, new = _lengths(c)
    totals = [x + n for x, n in zip(ctx, new)]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    t = start[-1]
    s["query_start"] = torch.tensor(start, dtype=torch.int32, device=DEVICE)
    s["max_new"], s["max_len"], s["scale"] = max(new), max(totals), c["dim"] ** -0.5
    if c["op"] != "paged":
        # the projections' packed output
        h, kv, d = c["heads"], c["kv_heads"], c["dim"]
        qkv = torch.randn((t, (h + 2 * kv) * d), device=DEVICE, generator=gen).to(torch.bfloat16)
        s["q"] = qkv[:, :h * d].view(t, h, d)
        s["k"] = qkv[:, h * d:(h + kv) * d].view(t, kv, d)
        s["v"] = qkv[:, (h + kv) * d:].view(t, kv, d)
    if c["op"] == "prompt":
        return s
    s["seq_lens"] = torch.tensor(totals, dtype=torch.int32, device=DEVICE)
    pages, s["table"] = _table(c, totals, gen)
    s["cache"], s["scales"] = _cache(pages, c, gen)
    if c["op"] == "paged":
        s["q"] = torch.randn((t, c["heads"], c["dim"]), device=DEVICE, generator=gen).to(torch.bfloat16)
        return s
    s["positions"] = torch.cat([torch.arange(x, x + n, device=DEVICE) for x, n in zip(ctx, new)])
    half = c["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)
    angle = torch.arange(8192, device=DEVICE, dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    y, rest = x[..., :rot], x[..., rot:]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, rest], -1)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, between LEAST and MOST."""
    fraction, power = torch.frexp(amax)                  # amax = fraction * 2^power, 448 = 0.875 * 2^9
    e = power - 8 - (fraction <= 0.875).int()
    return torch.where(amax == 0, LEAST, e.clamp(LEAST, MOST))


def _offsets_first(s):
    """The cache [pages, 2, offset, head, dim], a view."""
    return s["cache"] if s["case"]["layout"] == "NHD" else s["cache"].transpose(2, 3)


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    cos_sin = s["cos_sin"][s["positions"]][:, None]
    cos, sin = cos_sin[..., :c["rot"] // 2], cos_sin[..., c["rot"] // 2:]
    q = _rotate(s["q"].float(), cos, sin, c["interleaved"]).to(torch.bfloat16)
    k = _rotate(s["k"].float(), cos, sin, c["interleaved"])
    new = torch.stack([k, s["v"].float()], 1)                              # [T, 2, kv, D]
    t, start = new.shape[0], s["query_start"].long()
    token = torch.arange(t, device=DEVICE)
    request = torch.searchsorted(start, token, right=True) - 1
    first = s["seq_lens"].long() - (start[1:] - start[:-1])                # position of a request's first new token
    pos = first[request] + token - start[request]
    page = s["table"].long()[request, pos // c["page"]]
    old = s["scales"].int() - BIAS
    side_head = 2 * c["kv_heads"]
    top = torch.zeros((old.shape[0], side_head), device=DEVICE)
    top.scatter_reduce_(0, page[:, None].expand(-1, side_head), new.abs().amax(-1).view(t, -1), "amax")
    e = _exponent(top).view(old.shape)
    # what a page holds before the request's first new token stays, under a scale that covers both
    head_page = s["table"].long().gather(1, (first // c["page"])[:, None])[:, 0]
    held = first % c["page"]
    touched = torch.zeros(old.shape[0], dtype=torch.bool, device=DEVICE)
    touched[page] = True
    kept = torch.zeros_like(touched)
    kept[head_page] = held > 0
    e = torch.where(touched[:, None, None], torch.where(kept[:, None, None], torch.maximum(e, old), e), old)
    cache = _offsets_first(s)
    codes = cache[head_page]                                               # [B, 2, page, kv, D]
    shrink = torch.exp2((old - e)[head_page].float())[:, :, None, :, None]
    again = _e4m3(codes.view(torch.float8_e4m3fn).float() * shrink)
    live = torch.arange(c["page"], device=DEVICE) < held[:, None]
    cache[head_page] = torch.where(live[:, None, :, None, None], again, codes)
    cache[page, :, pos % c["page"]] = _e4m3(new * torch.exp2(-e[page].float())[..., None])
    s["scales"].copy_(e + BIAS)
    return {"q": q, "k": k.to(torch.bfloat16), "cache": s["cache"].view(torch.float8_e4m3fn), "scales": s["scales"]}


def _read(s, side, page, off):
    """fp32 values [B, K, kv_heads, dim] of one side at (page, off) [B, K]."""
    code = _offsets_first(s)[page, side, off]
    scale = torch.exp2(s["scales"][page, side].float() - BIAS)
    return code.view(torch.float8_e4m3fn).float() * scale[..., None]


def _softmax(score, see, values):
    """Weighted values and log-sum-exp of scores [..., rows, keys]; rows that see nothing give 0 and -inf."""
    score.masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    den = weight.sum(-1, keepdim=True)
    return torch.matmul(weight, values) / torch.where(den > 0, den, 1), (top + torch.log(den))[..., 0]


def _rows(s, ctx, count):
    """Queries [B, kv, n * g, D] of every request, padded to the longest, their positions, and the way back."""
    c = s["case"]
    b, n, g, kv = c["batch"], s["max_new"], c["heads"] // c["kv_heads"], c["kv_heads"]
    i = torch.arange(n, device=DEVICE)
    t = s["q"].shape[0]
    row = (s["query_start"][:-1].long()[:, None] + i).clamp(max=t - 1)
    q = s["q"][row].float().view(b, n, kv, g, c["dim"]).permute(0, 2, 1, 3, 4).reshape(b, kv, n * g, c["dim"])
    live = (i < count).reshape(-1)
    pick = torch.zeros(t + 1, dtype=torch.long, device=DEVICE)
    pick[torch.where(live, row.reshape(-1), t)] = torch.arange(b * n, device=DEVICE)

    def back(out, lse):
        out = out.view(b, kv, n, g, c["dim"]).permute(0, 2, 1, 3, 4).reshape(b * n, c["heads"], c["dim"])
        lse = lse.view(b, kv, n, g).permute(0, 2, 1, 3).reshape(b * n, c["heads"])
        return {"out": out[pick[:-1]].to(torch.bfloat16), "lse": lse[pick[:-1]]}

    return q, ctx + i, row, back


def _sees(c, pos, at, there):
    """Which positions [B, K] the queries at positions [B, n] see, as [B, 1, n * g, K]."""
    see = (pos[:, None] <= at[..., None]) & there[:, None]
    if c["window"]:
        see &= (pos[:, None] > at[..., None] - c["window"]) | (pos < c["sinks"])[:, None]
    return see.repeat_interleave(c["heads"] // c["kv_heads"], 1)[:, None]


def _plain_paged(s):
    c = s["case"]
    b, n = c["batch"], s["max_new"]
    total = s["seq_lens"].long()[:, None]
    count = (s["query_start"][1:] - s["query_start"][:-1]).long()[:, None]
    ctx = total - count
    # positions that some query of the request may see: the first tokens, then the window's range
    if c["window"]:
        first = (ctx - c["window"] + 1).clamp(min=0)
        near = first + torch.arange(min(s["max_len"], c["window"] + n - 1), device=DEVICE)
        far = torch.arange(c["sinks"], device=DEVICE).expand(b, -1)
        pos = torch.cat([far, near], 1)
        there = torch.cat([(far < first) & (far < total), near < total], 1)
    else:
        pos = torch.arange(s["max_len"], device=DEVICE).expand(b, -1)
        there = pos < total
    column = torch.where(there, pos // c["page"], 0)
    page = torch.where(there, s["table"].long().gather(1, column), 0)
    off = torch.where(there, pos % c["page"], 0)
    q, at, _, back = _rows(s, ctx, count)
    keys = _read(s, 0, page, off).permute(0, 2, 3, 1)                      # [B, kv, D, K]
    score = torch.matmul(q, keys) * s["scale"]
    del keys
    values = _read(s, 1, page, off).permute(0, 2, 1, 3)                    # [B, kv, K, D]
    return back(*_softmax(score, _sees(c, pos, at, there), values))


def _plain_prompt(s):
    c = s["case"]
    count = (s["query_start"][1:] - s["query_start"][:-1]).long()[:, None]
    q, at, row, back = _rows(s, torch.zeros_like(count), count)
    score = torch.matmul(q, s["k"][row].float().permute(0, 2, 3, 1)) * s["scale"]
    values = s["v"][row].float().permute(0, 2, 1, 3)
    return back(*_softmax(score, _sees(c, at, at, at < count), values))


def run(s):
    c = s["case"]
    if own:
        import fp8_quantized_paged_concat_gb300 as kvq
        if c["op"] == "append":
            q, k = kvq.kvq_rope_append_fp8_per_head(
                s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["query_start"], s["seq_lens"], s["table"],
                s["cache"], s["scales"], s["max_new"], interleaved=c["interleaved"], layout=c["layout"])
            return {"q": q, "k": k, "cache": s["cache"].view(torch.float8_e4m3fn), "scales": s["scales"]}
        if c["op"] == "paged":
            out, lse = kvq.kvq_window_attention_fp8_per_head(
                s["q"], s["query_start"], s["seq_lens"], s["table"], s["cache"], s["scales"], s["scale"], s["max_new"],
                s["max_len"], window=c["window"], num_sinks=c["sinks"], layout=c["layout"])
            return {"out": out, "lse": lse}
        out, lse = kvq.kvq_prompt_attention(s["q"], s["k"], s["v"], s["query_start"], s["scale"], s["max_new"],
                                            window=c["window"], num_sinks=c["sinks"])
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "paged":
        return _plain_paged(s)
    return _plain_prompt(s)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _code_values():
    """The value of each e4m3 code: sign, 4 exponent bits, 3 fraction bits."""
    v = []
    for x in range(256):
        e, f = (x >> 3) & 15, x & 7
        a = math.nan if e == 15 and f == 7 else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append(-a if x & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=DEVICE)


def _exact_append(s):
    """q and k; the cache and its scales are what the definition's fp32 steps make of them, with no value of their own."""
    c = s["case"]
    half = c["rot"] // 2
    table = s["cos_sin"].double()[s["positions"]]
    got = []
    for x in (s["q"], s["k"]):
        y = x.double()
        z = y.clone()
        for d in range(half):
            a, b = (2 * d, 2 * d + 1) if c["interleaved"] else (d, d + half)
            co, si = table[:, d, None], table[:, half + d, None]
            z[..., a] = y[..., a] * co - y[..., b] * si
            z[..., b] = y[..., b] * co + y[..., a] * si
        got.append(z)
    return {"q": got[0], "k": got[1], "cache": None, "scales": None}


def _exact_attention(s):
    c = s["case"]
    dim, kv, g = c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    starts = s["query_start"].tolist()
    t = s["q"].shape[0]
    out = torch.zeros((t, kv, g, dim), dtype=torch.float64, device=DEVICE)
    lse = torch.full((t, kv, g), -math.inf, dtype=torch.float64, device=DEVICE)
    values = _code_values()
    for b in range(len(starts) - 1):
        t0, n = starts[b], starts[b + 1] - starts[b]
        ctx = int(s["seq_lens"][b]) - n if c["op"] == "paged" else 0
        for h in range(kv):
            if c["op"] == "prompt":
                sides = [s[x][t0:t0 + n, h].double() for x in "kv"]
            else:
                pos = torch.arange(ctx + n, device=DEVICE)
                page, off = s["table"][b].long()[pos // c["page"]], pos % c["page"]
                sides = []
                for side in (0, 1):
                    code = s["cache"][page, side, off, h] if c["layout"] == "NHD" else s["cache"][page, side, h, off]
                    sides.append(values[code.long()] * torch.pow(2.0, s["scales"][page, side, h].double() - BIAS)[:, None])
            q = s["q"][t0:t0 + n, h * g:(h + 1) * g].double()
            for i in range(0, n, 2048):
                m = min(2048, n - i)
                hi = ctx + i + m                                           # keys before hi, from lo on, and the first
                lo = max(0, ctx + i - c["window"] + 1) if c["window"] else 0
                pos = torch.cat([torch.arange(min(c["sinks"], lo), device=DEVICE), torch.arange(lo, hi, device=DEVICE)])
                at = (ctx + i + torch.arange(m, device=DEVICE))[:, None]
                see = pos <= at
                if c["window"]:
                    see = see & ((at - pos < c["window"]) | (pos < c["sinks"]))
                k, v = sides[0][pos], sides[1][pos]
                for j in range(g):
                    x = (q[i:i + m, j] @ k.T) * s["scale"]
                    x[~see] = -math.inf
                    top = x.max(1).values
                    w = (x - top[:, None]).exp_()
                    out[t0 + i:t0 + i + m, h, j] = (w @ v) / w.sum(1, keepdim=True)
                    lse[t0 + i:t0 + i + m, h, j] = top + w.sum(1).log()
    return {"out": out.flatten(1, 2), "lse": lse.flatten(1, 2)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
