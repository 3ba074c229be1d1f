"""Plain 64-bit references for serving from the per-head NVFP4 cache (numpy,
CPU, written from the definitions), and the inputs its tests share."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(code):
    """Values of e4m3 codes (0x7F and 0xFF are NaN)."""
    code = np.asarray(code, np.int64)
    s, e, m = np.where(code & 0x80, -1.0, 1.0), (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    return s * np.where((e == 15) & (m == 7), np.nan, v)


def bf16(x):
    """float64 values of bf16 bit patterns."""
    return (np.asarray(x).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16(x):
    """fp32 values -> bf16 bit patterns, round to nearest even."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


class Cache:
    """A per-head cache on the host: raw bytes [layers, pages, 2, region]."""

    def __init__(self, layers, pages, block, heads, dim, layout, rng):
        self.block, self.heads, self.dim, self.layout = block, heads, dim, layout
        self.cut = block * heads * dim // 2
        region = self.cut + block * heads * dim // 16
        self.raw = rng.integers(0, 256, (layers, pages, 2, region), dtype=np.uint8)
        # scales: mostly ordinary, a few zero, subnormal or negative
        n = (layers, pages, 2, region - self.cut)
        sf = rng.integers(0x1C, 0x34, n, dtype=np.uint8)
        odd = rng.random(n)
        sf = np.where(odd < 0.02, 0, np.where(odd < 0.04, rng.integers(1, 8, n), np.where(odd < 0.06, sf | 0x80, sf)))
        self.raw[..., self.cut:] = sf

    def shape(self):
        full = self.dim // 2 + self.dim // 16
        inner = (self.block, self.heads, full) if self.layout == "NHD" else (self.heads, self.block, full)
        return self.raw.shape[:3] + inner

    def row(self, off, head):
        return off * self.heads + head if self.layout == "NHD" else head * self.block + off

    def spans(self, off, head):
        """Byte ranges of an entry inside its (page, side): data, scales."""
        r = self.row(off, head)
        d, s = self.dim // 2, self.dim // 16
        return slice(r * d, r * d + d), slice(self.cut + r * s, self.cut + r * s + s)

    def entry(self, page, side, off, head, layer=0):
        a, b = self.spans(off, head)
        raw = self.raw[layer, page, side]
        code = np.stack([raw[a] & 15, raw[a] >> 4], -1).reshape(-1)
        return E2M1[code] * np.repeat(e4m3(raw[b]), 16)


def keys_of(cache, table, head, positions):
    """Decoded (K, V) of the positions; None where the page is out of range."""
    pages = cache.raw.shape[1]
    out = []
    for p in positions:
        col = p // cache.block
        page = table[col] if col < len(table) else -1
        out.append(None if not 0 <= page < pages else
                   (cache.entry(page, 0, p % cache.block, head), cache.entry(page, 1, p % cache.block, head)))
    return out


def attention(cache, q, query_start, seq_lens, table, k_scale, v_scale, scale, window=0, sinks=0, tree=None):
    """out, lse and the per-element tolerances of the kernel's arithmetic.

    Per row: e_s bounds the score error (an fp32 sum of D exact products, and
    two more roundings of its scaling; q itself is exact in f16 down to 2^-28
    of the row's largest value, below which a value is off by at most 2^-39
    of it), a weight carries one f16 rounding (2^-11), the exponential 2^-20,
    an f16 weight below the normal range is off by at most 2^-31 of the
    largest one, and the two fp32 sums over n keys n 2^-24 each."""
    T, H, D = q.shape
    KH = cache.heads
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    tol_o, tol_l = np.zeros((T, H, D)), np.zeros((T, H))
    for b, length in enumerate(seq_lens):
        t0, t1 = query_start[b], query_start[b + 1]
        n = t1 - t0
        for kh in range(KH):
            kv = keys_of(cache, table[b], kh, range(max(0, length)))
            for i in range(n):
                p = length - n + i
                if tree is not None:
                    base = length - n
                    see = [j for j in range(max(0, length))
                           if kv[j] is not None and (j < base or (int(tree[t0 + i][(j - base) // 64]) >> ((j - base) % 64)) & 1)]
                else:
                    see = [j for j in range(max(0, length)) if kv[j] is not None and j <= p
                           and (window <= 0 or j > p - window or j < sinks)]
                if not see:
                    continue
                K = np.stack([kv[j][0] for j in see])
                V = np.stack([kv[j][1] for j in see])
                V = np.where(np.isnan(V), 0.0, V)
                for h in range(kh * (H // KH), (kh + 1) * (H // KH)):
                    x = q[t0 + i, h]
                    s = (K @ x) * (scale * k_scale)
                    m = s.max()
                    w = np.exp(s - m)
                    out[t0 + i, h] = v_scale * (w @ V) / w.sum()
                    lse[t0 + i, h] = m + np.log(w.sum())
                    size = abs(scale * k_scale) * (np.abs(K) @ np.abs(x)).max()
                    lost = abs(scale * k_scale) * np.abs(K).sum(1).max() * np.abs(x).max() * 2.0 ** -39
                    e_s = (D + 4) * 2.0 ** -24 * size + lost
                    sums = (len(see) + 32) * 2.0 ** -24
                    mean = abs(v_scale) * (w @ np.abs(V)) / w.sum()
                    tiny = abs(v_scale) * len(see) * 2.0 ** -31 * np.abs(V).max(0)
                    tol_o[t0 + i, h] = (2.0 ** -11 + 2 * e_s + 2 * sums + 2.0 ** -18) * mean + tiny \
                        + 2.0 ** -8 * np.abs(out[t0 + i, h]) + 1e-30
                    tol_l[t0 + i, h] = e_s + sums + 2.0 ** -19 + 2.0 ** -21 * abs(lse[t0 + i, h])
    return out, lse, tol_o, tol_l


def norm_rope(x, w, positions, cos_sin, rot, eps, interleaved):
    """Result and tolerance: fp32 arithmetic ((D + 16) roundings of 2^-24 on
    each product that makes a value up) and one bf16 rounding (2^-8)."""
    D = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    z, size = y.copy(), np.abs(y)
    half = rot // 2
    c = cos_sin[positions][:, None, :half].astype(np.float64)
    s = cos_sin[positions][:, None, half:rot].astype(np.float64)
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + (1 if interleaved else half)
    a, b = y[..., ia], y[..., ib]
    z[..., ia], z[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia], size[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return z, (D + 16) * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(z) + 1e-37


def compact(cache, query_start, seq_lens, accepted, accepted_lens, table):
    """The cache after the accepted drafts moved (all reads before all writes)."""
    before, after = cache.raw, cache.raw.copy()
    pages = before.shape[1]
    for b, length in enumerate(seq_lens):
        n = query_start[b + 1] - query_start[b]
        m = accepted_lens[b]
        base = length - n
        if n < 0 or base < 0 or not 0 <= m <= accepted.shape[1]:
            continue
        a = [int(v) for v in accepted[b, :m]]
        if any(not 0 <= v < n for v in a) or any(v <= u for u, v in zip(a, a[1:])):
            continue
        for i, v in enumerate(a):
            src, dst = base + v, base + i
            where = []
            for p in (src, dst):
                col = p // cache.block
                where.append(table[b, col] if col < table.shape[1] else -1)
            if not all(0 <= w < pages for w in where):
                continue
            for h in range(cache.heads):
                for x, y in zip(cache.spans(src % cache.block, h), cache.spans(dst % cache.block, h)):
                    after[:, where[1], :, y] = before[:, where[0], :, x]
    return after
