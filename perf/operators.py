"""Measured cases of the operators that serve a model from the per-head NVFP4 K/V cache.

Four operators, each in its plain form (torch, 32 bits) and, with ``own``, as
the calls a user makes of this framework:

  norm_rope  RMS norm of every query and key head, and the position rotation,
             on the projections' output (before the keys go into the cache);
  window     attention over the paged cache: causal, with a sliding window
             and a few first tokens that stay visible, for single decoded
             tokens and for chunks of new tokens;
  tree       attention of drafted tokens that form a tree (each sees the
             context and the drafts its mask names) over the same cache;
  compact    after the drafts are checked: the accepted ones' entries moved
             to consecutive positions, in every layer's cache.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
CODES = [v for v in E2M1] + [-v for v in E2M1]          # value of each 4-bit code
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _norm(name, tokens, heads, kv_heads, dim, rot, interleaved=False, max_pos=65536):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "interleaved": interleaved, "max_pos": max_pos}


def _attn(name, op, batch, new, ctx_lo, ctx_hi, heads, kv_heads, dim, page, layout, window=0, sinks=0, ragged=False):
    return {"name": name, "op": op, "batch": batch, "new": new, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "layout": layout, "window": window, "sinks": sinks,
            "ragged": ragged}


def _compact(name, layers, batch, drafts, depth, ctx_lo, ctx_hi, kv_heads, dim, page, layout):
    return {"name": name, "op": "compact", "layers": layers, "batch": batch, "drafts": drafts, "depth": depth,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "kv_heads": kv_heads, "dim": dim, "page": page, "layout": layout}


def listed():
    return [
        # one decode step of a batch of 64: a launch-bound call
        _norm("norm_rope decode 64", 64, 32, 8, 128, 128),
        # a prefill chunk: one read and one write of every query and key
        _norm("norm_rope prefill 16384", 16384, 32, 8, 128, 128),
        # one user's decode step on a layer with a short window: latency
        _attn("window decode 1", "window", 1, 1, 20000, 20000, 64, 8, 128, 16, "NHD", 1024, 4),
        # a full decode batch on a windowed layer
        _attn("window decode 128", "window", 128, 1, 4096, 16384, 32, 8, 128, 16, "NHD", 4096, 4),
        # the same on a layer without a window, over the repository's long contexts
        _attn("window decode 32 full", "window", 32, 1, 7378, 34474, 32, 8, 128, 16, "NHD"),
        # chunked prefill of four requests on a windowed layer
        _attn("window prefill 4x4096", "window", 4, 4096, 0, 8192, 32, 8, 128, 16, "NHD", 4096, 4),
        # odd sizes: 7 query heads per key head, ragged chunks, pages of 24, head-major cache
        _attn("window prefill odd", "window", 7, 777, 0, 3000, 21, 3, 64, 24, "HND", 333, 17, True),
        # one user's draft tree
        _attn("tree 1x24", "tree", 1, 24, 8000, 8000, 32, 8, 128, 16, "NHD"),
        # a batch of draft trees over long contexts
        _attn("tree 32x64", "tree", 32, 64, 7378, 34474, 32, 8, 128, 16, "NHD"),
        # wide heads, ragged trees of up to 100 drafts (two mask words), head-major cache
        _attn("tree ragged dim 256", "tree", 5, 100, 100, 5000, 16, 2, 256, 32, "HND", 0, 0, True),
        # acceptance of one user's drafts in one layer
        _compact("compact 1 layer x 4", 1, 4, 16, 6, 40, 400, 8, 128, 16, "NHD"),
        # acceptance of a batch's drafts in all layers
        _compact("compact 32 layers x 64", 32, 64, 64, 12, 40, 400, 8, 128, 16, "NHD"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        # no dearer than the largest listed case, in the plain form's memory too
        if w["bytes"] <= 7.5e8 and w["flops"] <= 1.0e12 and _plain_values(c) <= 9e9:
            return c


def _draw(rng):
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8, 8])
    heads = kv * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
    page = rng.choice([16, 16, 32, 48, 64])
    layout = rng.choice(["NHD", "HND"])
    kind = rng.choice(["norm_rope", "decode", "decode", "prefill", "prefill", "tree", "tree", "compact"])
    if kind == "norm_rope":
        c = _norm("", _log(rng, 1, 16384), heads, kv, dim, rng.choice([dim, dim, dim // 2, 32]), rng.random() < 0.3,
                  _log(rng, 1024, 131072))
    elif kind == "compact":
        drafts = _log(rng, 2, 128)
        c = _compact("", _log(rng, 1, 32), _log(rng, 1, 64), drafts, rng.randint(1, min(drafts, 16)), 0,
                     _log(rng, 16, 400), kv, dim, page, layout)
    else:
        hi = _log(rng, 16, 34000)
        lo = rng.randint(0, hi)
        if kind == "decode":
            window = rng.choice([0, 0, _log(rng, 1, 8192)])
            c = _attn("", "window", _log(rng, 1, 128), 1, lo, hi, heads, kv, dim, page, layout, window,
                      rng.choice([0, 4, rng.randint(1, 128)]))
        elif kind == "prefill":
            window = rng.choice([0, _log(rng, 16, 8192)])
            c = _attn("", "window", _log(rng, 1, 16), _log(rng, 2, 4096), lo, hi, heads, kv, dim, page, layout, window,
                      rng.choice([0, 4, rng.randint(1, 128)]), rng.random() < 0.5)
        else:
            c = _attn("", "tree", _log(rng, 1, 32), _log(rng, 2, 128), lo, hi, heads, kv, dim, page, layout, 0, 0,
                      rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(c):
    """Contexts and new tokens of each request: fixed by the case, not by the seed."""
    r = random.Random("%s %s %s %s" % (c["batch"], c["ctx_lo"], c["ctx_hi"], c.get("new", c.get("drafts"))))
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["batch"])]
    most = c.get("new", c.get("drafts"))
    new = [r.randint(1, most) if c.get("ragged") and b else most for b in range(c["batch"])]
    return ctx, new


def _accepted(c):
    """Accepted drafts of each request: increasing draft numbers, fixed by the case."""
    r = random.Random("accepted %s %s %s" % (c["batch"], c["drafts"], c["depth"]))
    return [sorted(r.sample(range(c["drafts"]), r.randint(0, c["depth"]))) for _ in range(c["batch"])]


def _visible(c, ctx, new):
    """(keys read at least once, (query, key) pairs) of one request."""
    total = ctx + new
    if c["op"] == "tree":
        return total, new * ctx + new * (new + 1) // 2       # a tree's masks keep at most the triangle
    w, ns = c["window"], c["sinks"]
    pairs = keys = 0
    first = total
    for i in range(new):
        p = ctx + i
        lo = max(0, p - w + 1) if w > 0 else 0
        first = min(first, lo)
        pairs += p + 1 - lo + min(ns, lo)
    keys = total - first + min(ns, first)
    return keys, pairs


def _plain_values(c):
    """Scores of the plain form, all at once."""
    if c["op"] not in ("window", "tree"):
        return 0
    ctx, new = _lengths(c)
    keys = c["ctx_hi"] + c["new"]
    if c["window"]:
        keys = min(keys, c["window"] + c["new"]) + c["sinks"]
    return c["batch"] * max(c["heads"] * c["new"] * keys, 2 * c["kv_heads"] * c["dim"] * keys)


def work(c):
    if c["op"] == "norm_rope":
        values = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 4 * values + c["tokens"] * (8 + 4 * c["rot"]), "flops": 6 * values}
    row = c["dim"] // 2 + c["dim"] // 16                     # one side of one head of one position
    if c["op"] == "compact":
        moved = sum(a != i for acc in _accepted(c) for i, a in enumerate(acc))
        return {"bytes": max(1, moved) * 2 * 2 * c["layers"] * c["kv_heads"] * row, "flops": 0}
    ctx, new = _lengths(c)
    seen = [_visible(c, x, n) for x, n in zip(ctx, new)]
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    tokens = sum(new)
    return {"bytes": keys * c["kv_heads"] * 2 * row + tokens * c["heads"] * (4 * c["dim"] + 4)
            + sum((x + n + c["page"] - 1) // c["page"] for x, n in zip(ctx, new)) * 4,
            "flops": 4 * c["dim"] * c["heads"] * pairs}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _cache(layers, pages, c, gen):
    """A cache whose entries look like quantized normals: codes with the
    frequencies of a normal whose largest of 16 is 6, scales around 0.3."""
    full = c["dim"] // 2 + c["dim"] // 16
    side = c["page"] * c["kv_heads"] * full
    data = c["page"] * c["kv_heads"] * (c["dim"] // 2)
    cut = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEVICE)
    x = 3.4 * torch.special.ndtri((torch.arange(256, device=DEVICE, dtype=torch.float32) + 0.5) / 256)
    nibble = torch.bucketize(x.abs(), cut) + 8 * (x < 0)
    pair = (nibble[:, None] * 16 + nibble[None, :]).reshape(-1).to(torch.uint8)
    cache = torch.empty((layers * pages * 2, side), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 28) // side)
    for i in range(0, cache.shape[0], step):
        n = min(step, cache.shape[0] - i)
        at = torch.randint(0, 65536, (n, data), device=DEVICE, generator=gen, dtype=torch.int32)
        cache[i:i + n, :data] = pair.index_select(0, at.reshape(-1)).view(n, data)
        cache[i:i + n, data:] = torch.randint(0x26, 0x2E, (n, side - data), device=DEVICE, generator=gen,
                                              dtype=torch.uint8)
    inner = (c["page"], c["kv_heads"], full) if c["layout"] == "NHD" else (c["kv_heads"], c["page"], full)
    return cache.view(layers, pages, 2, *inner)


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


def _tree_mask(new, words, rng):
    """Each draft sees itself and its ancestors; a draft's parent is one of the eight before it or the context."""
    rows = []
    for n in new:
        seen = []
        for i in range(n):
            parent = rng.randint(max(-1, i - 8), i - 1)
            seen.append((1 << i) | (seen[parent] if parent >= 0 else 0))
        for m in seen:
            w = [(m >> (64 * j)) & (2 ** 64 - 1) for j in range(words)]
            rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in w])
    return torch.tensor(rows, dtype=torch.int64).to(DEVICE)


def prepare(c, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(1000 + seed)
    s = {"case": c}
    if c["op"] == "norm_rope":
        t, width = c["tokens"], (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
        # the projections' packed output; its values side is not touched here
        s["qkv"] = (torch.randn((t, width), device=DEVICE, generator=gen) * 1.7).to(torch.bfloat16)
        s["q"] = s["qkv"][:, :c["heads"] * c["dim"]].view(t, c["heads"], c["dim"])
        s["k"] = s["qkv"][:, c["heads"] * c["dim"]:-c["kv_heads"] * c["dim"]].view(t, c["kv_heads"], c["dim"])
        for w in ("q_weight", "k_weight"):
            s[w] = (1 + 0.2 * torch.randn(c["dim"], device=DEVICE, generator=gen)).to(torch.bfloat16)
        s["positions"] = torch.randint(0, c["max_pos"], (t,), device=DEVICE, generator=gen)
        half = c["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)
        angle = torch.arange(c["max_pos"], device=DEVICE, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        return s
    ctx, new = _lengths(c)
    totals = [x + n for x, n in zip(ctx, new)]
    pages, s["table"] = _table(c, totals, gen)
    s["seq_lens"] = torch.tensor(totals, dtype=torch.int32, device=DEVICE)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s["query_start"] = torch.tensor(start, dtype=torch.int32, device=DEVICE)
    s["max_new"], s["max_len"] = max(new), max(totals)
    if c["op"] == "compact":
        s["cache"] = _cache(c["layers"], pages, c, gen)
        acc = _accepted(c)
        s["accepted"] = torch.tensor([a + [0] * (c["depth"] - len(a)) for a in acc], dtype=torch.int32).to(DEVICE)
        s["accepted_lens"] = torch.tensor([len(a) for a in acc], dtype=torch.int32, device=DEVICE)
        return s
    s["cache"] = _cache(1, pages, c, gen)[0]
    s["q"] = torch.randn((start[-1], c["heads"], c["dim"]), device=DEVICE, generator=gen).to(torch.bfloat16)
    s["k_scale"] = torch.tensor([0.9], device=DEVICE)
    s["v_scale"] = torch.tensor([1.1], device=DEVICE)
    s["scale"] = c["dim"] ** -0.5
    if c["op"] == "tree":
        s["tree_mask"] = _tree_mask(new, (s["max_new"] + 63) // 64, random.Random(seed))
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


def _plain_norm_rope(s):
    c = s["case"]
    cos_sin = s["cos_sin"][s["positions"]][:, None]
    cos, sin = cos_sin[..., :c["rot"] // 2], cos_sin[..., c["rot"] // 2:]
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s[name + "_weight"].float()
        out[name] = _rotate(x, cos, sin, c["interleaved"]).to(torch.bfloat16)
    return out


def _views(cache, c):
    """(codes, scales) of a cache [..., page count, 2, ...], offsets before heads."""
    lead = cache.shape[:-3]
    flat = cache.reshape(*lead, -1)
    cut = c["page"] * c["kv_heads"] * c["dim"] // 2
    inner = (c["page"], c["kv_heads"]) if c["layout"] == "NHD" else (c["kv_heads"], c["page"])
    data = flat[..., :cut].unflatten(-1, (*inner, c["dim"] // 2))
    scales = flat[..., cut:].unflatten(-1, (*inner, c["dim"] // 16))
    return (data, scales) if c["layout"] == "NHD" else (data.transpose(-3, -2), scales.transpose(-3, -2))


def _read(s, side, page, off):
    """fp32 values [B, K, kv_heads, dim] of one side at (page, off) [B, K], without the tensor's scale."""
    c = s["case"]
    data, scales = _views(s["cache"], c)
    code = data[page, side, off]
    code = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    lut = torch.tensor(CODES, device=DEVICE)
    x = lut.index_select(0, code.reshape(-1).int()).view(*code.shape[:-1], c["dim"] // 16, 16)
    sf = scales[page, side, off].contiguous().view(torch.float8_e4m3fn).float()
    return (x * sf[..., None]).flatten(-2)


def _plain_attention(s):
    c = s["case"]
    b, n, g, kv = c["batch"], s["max_new"], c["heads"] // c["kv_heads"], c["kv_heads"]
    total = s["seq_lens"].long()[:, None]
    count = (s["query_start"][1:] - s["query_start"][:-1]).long()[:, None]
    ctx = total - count
    # positions that some query of the request may see: the first tokens, then the window's range
    if c["window"]:
        first = (ctx - c["window"] + 1).clamp(min=0)
        span = min(s["max_len"], c["window"] + n - 1)
        near = first + torch.arange(span, device=DEVICE)
        far = torch.arange(c["sinks"], device=DEVICE).expand(b, -1)
        pos = torch.cat([far, near], 1)
        there = torch.cat([(far < first) & (far < total), near < total], 1)
    else:
        pos = torch.arange(s["max_len"], device=DEVICE).expand(b, -1)
        there = pos < total
    column = torch.where(there, pos // c["page"], 0)
    page = torch.where(there, s["table"].long().gather(1, column), 0)
    off = torch.where(there, pos % c["page"], 0)
    keys = _read(s, 0, page, off).permute(0, 2, 3, 1)                      # [B, kv, D, K]
    i = torch.arange(n, device=DEVICE)
    at = ctx + i                                                           # [B, n]: the queries' positions
    row = (s["query_start"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(b, n, kv, g, c["dim"]).permute(0, 2, 1, 3, 4).reshape(b, kv, n * g, c["dim"])
    score = torch.matmul(q, keys) * (s["scale"] * s["k_scale"])
    del keys
    if c["op"] == "tree":
        draft = (pos - ctx).clamp(min=0)[:, None]                           # [B, 1, K]
        words = s["tree_mask"][row]                                        # [B, n, W]
        word = words.gather(2, (draft // 64).clamp(max=words.shape[2] - 1).expand(-1, n, -1))
        see = (pos < ctx)[:, None] | ((word >> (draft % 64)) & 1).bool()
    else:
        see = pos[:, None] <= at[..., None]
        if c["window"]:
            see &= (pos[:, None] > at[..., None] - c["window"]) | (pos < c["sinks"])[:, None]
    see = (see & there[:, None]).repeat_interleave(g, 1)[:, None]
    score.masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score.sub_(torch.where(top == -math.inf, 0, top)))
    del score
    den = weight.sum(-1, keepdim=True)
    values = _read(s, 1, page, off).permute(0, 2, 1, 3)                    # [B, kv, K, D]
    out = torch.matmul(weight, values) / torch.where(den > 0, den, 1) * s["v_scale"]
    lse = (top + torch.log(den))[..., 0]
    live = (i < count).reshape(-1)                                         # request by request, token by token
    out = out.view(b, kv, n, g, c["dim"]).permute(0, 2, 1, 3, 4).reshape(b * n, c["heads"], c["dim"])
    lse = lse.view(b, kv, n, g).permute(0, 2, 1, 3).reshape(b * n, c["heads"])
    pick = torch.zeros(s["q"].shape[0] + 1, dtype=torch.long, device=DEVICE)
    pick[torch.where(live, row.reshape(-1), s["q"].shape[0])] = torch.arange(b * n, device=DEVICE)
    return {"out": out[pick[:-1]].to(torch.bfloat16), "lse": lse[pick[:-1]]}


def _plain_compact(s):
    c = s["case"]
    data, scales = _views(s["cache"], c)
    i = torch.arange(c["depth"], device=DEVICE)
    count = (s["query_start"][1:] - s["query_start"][:-1]).long()[:, None]
    ctx = s["seq_lens"].long()[:, None] - count
    last = count - 1
    to = ctx + torch.minimum(i, last)
    src = torch.where(i < s["accepted_lens"][:, None], ctx + s["accepted"], to)
    table = s["table"].long()
    at = (table.gather(1, to // c["page"]), to % c["page"])
    whence = (table.gather(1, src // c["page"]), src % c["page"])
    for v in (data, scales):
        moved = v[:, whence[0], :, whence[1]]
        v[:, at[0], :, at[1]] = moved
    return {"cache": s["cache"]}


def run(s):
    c = s["case"]
    if own:
        import fp8_quantized_paged_concat_gb300 as kvq
        if c["op"] == "norm_rope":
            q, k = kvq.kvq_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["cos_sin"], EPS,
                                        interleaved=c["interleaved"])
            return {"q": q, "k": k}
        if c["op"] == "window":
            out, lse = kvq.kvq_window_attention_nvfp4_per_head(
                s["q"], s["query_start"], s["seq_lens"], s["table"], s["cache"], s["k_scale"], s["v_scale"], s["scale"],
                s["max_new"], s["max_len"], window=c["window"], num_sinks=c["sinks"], layout=c["layout"])
            return {"out": out, "lse": lse}
        if c["op"] == "tree":
            out, lse = kvq.kvq_tree_attention_nvfp4_per_head(
                s["q"], s["query_start"], s["seq_lens"], s["tree_mask"], s["table"], s["cache"], s["k_scale"],
                s["v_scale"], s["scale"], s["max_new"], s["max_len"], layout=c["layout"])
            return {"out": out, "lse": lse}
        kvq.kvq_compact_drafts_nvfp4_per_head(s["cache"], s["query_start"], s["seq_lens"], s["accepted"],
                                              s["accepted_lens"], s["table"], layout=c["layout"])
        return {"cache": s["cache"]}
    if c["op"] == "norm_rope":
        return _plain_norm_rope(s)
    if c["op"] == "compact":
        return _plain_compact(s)
    return _plain_attention(s)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_norm_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    table = s["cos_sin"].double()[s["positions"]]
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        y = y / (y.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt() * w.double()
        z = y.clone()
        for d in range(half):
            a, b = (2 * d, 2 * d + 1) if c["interleaved"] else (d, d + half)
            co, si = table[:, d, None], table[:, half + d, None]
            z[..., a] = y[..., a] * co - y[..., b] * si
            z[..., b] = y[..., b] * co + y[..., a] * si
        got.append(z)
    return {"q": got[0], "k": got[1]}


def _exact_attention(s):
    c = s["case"]
    dim, kv, g, bs = c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"], c["page"]
    pairs = torch.tensor([[CODES[x & 15], CODES[x >> 4]] for x in range(256)], dtype=torch.float64, device=DEVICE)
    sides = s["cache"].flatten(2)
    cut = bs * kv * dim // 2
    starts, totals = s["query_start"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros((s["q"].shape[0], kv, g, dim), dtype=torch.float64, device=DEVICE)
    lse = torch.full((s["q"].shape[0], kv, g), -math.inf, dtype=torch.float64, device=DEVICE)
    ks, vs = s["k_scale"].double(), s["v_scale"].double()
    for b, total in enumerate(totals):
        n, t0 = starts[b + 1] - starts[b], starts[b]
        ctx = total - n
        pos = torch.arange(total, device=DEVICE)
        at = ctx + torch.arange(n, device=DEVICE)[:, None]
        if c["op"] == "tree":
            see = (pos < ctx).expand(n, -1).clone()
            for j in range(n):
                see[:, ctx + j] = ((s["tree_mask"][t0:t0 + n, j // 64] >> (j % 64)) & 1).bool()
        else:
            see = pos <= at
            if c["window"]:
                see = see & ((at - pos < c["window"]) | (pos < c["sinks"]))
        some = see.any(0)
        pos, see = pos[some], see[:, some]
        page, off = s["table"][b].long()[pos // bs], pos % bs
        for h in range(kv):
            row = off * kv + h if c["layout"] == "NHD" else h * bs + off
            kvs = []
            for side in (0, 1):
                r = sides[page, side]
                code = r.gather(1, row[:, None] * (dim // 2) + torch.arange(dim // 2, device=DEVICE))
                sf = r.gather(1, cut + row[:, None] * (dim // 16) + torch.arange(dim // 16, device=DEVICE))
                x = pairs[code.long()].reshape(-1, dim // 16, 16)
                kvs.append((x * sf.view(torch.float8_e4m3fn).double()[..., None]).reshape(-1, dim))
                del r
            q = s["q"][t0:t0 + n, h * g:(h + 1) * g].double()
            p = torch.einsum("ngd,kd->ngk", q, kvs[0]) * (s["scale"] * ks)
            p = p.masked_fill(~see[:, None], -math.inf)
            lse[t0:t0 + n, h] = torch.logsumexp(p, -1)
            p = torch.softmax(p, -1)
            out[t0:t0 + n, h] = torch.einsum("ngk,kd->ngd", p, kvs[1]) * vs
    return {"out": out.flatten(1, 2), "lse": lse.flatten(1)}


def exact(c, seed):
    if c["op"] == "compact":
        return None                                          # bytes: compared whole with the plain form's
    s = prepare(c, seed)
    return _exact_norm_rope(s) if c["op"] == "norm_rope" else _exact_attention(s)
