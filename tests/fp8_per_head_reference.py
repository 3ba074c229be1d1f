"""Plain references for serving from the per-head e4m3 cache and for attention
over whole prompts (numpy, CPU, written from the definitions): the append in
the definition's fp32 steps, attention in 64 bits with tolerances derived from
the kernels' arithmetic, and the inputs the tests share."""
import numpy as np

from per_head_reference import bf16, e4m3, to_bf16

BIAS, LEAST, MOST = 127, -60, 60

# e4m3 magnitudes in ascending order: code c has magnitude MAGNITUDE[c] (0x7F is NaN)
MAGNITUDE = e4m3(np.arange(127))


def to_e4m3(x):
    """fp32 values -> e4m3 codes: nearest, ties to the even code, saturating, NaN 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    hi = np.clip(np.searchsorted(MAGNITUDE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - MAGNITUDE[lo], MAGNITUDE[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def exponent(amax):
    """The least e in [LEAST, MOST] with amax <= 448 * 2^e."""
    for e in range(LEAST, MOST):
        if float(amax) <= 448.0 * 2.0 ** e:
            return e
    return MOST


class Cache:
    """A per-head e4m3 cache on the host: codes [pages, 2, block, heads, dim]
    in offsets-first order, scales [pages, 2, heads]."""

    def __init__(self, pages, block, heads, dim, layout, rng, exponents=(-9, -3)):
        self.block, self.heads, self.dim, self.layout = block, heads, dim, layout
        self.codes = rng.integers(0, 256, (pages, 2, block, heads, dim), dtype=np.uint8)
        self.codes[(self.codes & 0x7F) == 0x7F] = 0x38               # no NaN
        self.scales = (rng.integers(exponents[0], exponents[1] + 1, (pages, 2, heads)) + BIAS).astype(np.uint8)

    def raw(self):
        """The codes in the layout's order."""
        return np.ascontiguousarray(self.codes if self.layout == "NHD" else self.codes.swapaxes(2, 3))

    def from_raw(self, raw):
        return raw if self.layout == "NHD" else raw.swapaxes(2, 3)

    def values(self, page, side):
        """float64 [block, heads, dim] of a page's side."""
        e = np.clip(self.scales[page, side].astype(int) - BIAS, LEAST, MOST)
        return e4m3(self.codes[page, side]) * 2.0 ** e[:, None]


def rotate(x, c, s, interleaved):
    """fp32 [..., D] rotated by cosines and sines [..., rot / 2], one rounding per product and sum."""
    x, c, s = (np.asarray(v, np.float32) for v in (x, c, s))
    half = c.shape[-1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def append(cache, q, k, v, positions, cos_sin, start, lens, table, interleaved, q_out, k_out):
    """Appends in place; q, k, v, q_out, k_out are bf16 bits, the outputs written in place.  Returns the status bits."""
    half = cos_sin.shape[1] // 2
    status = 0
    pages = cache.codes.shape[0]
    for b, n_len in enumerate(lens):
        t0, t1 = start[b], start[b + 1]
        n, length = t1 - t0, max(0, n_len)
        if t0 < 0 or n < 0 or t1 > q.shape[0] or n > length:
            status |= 2
            continue
        by_page = {}
        for i in range(n):
            t, p = t0 + i, length - n + i
            live = 0 <= positions[t] < cos_sin.shape[0]
            col, off = p // cache.block, p % cache.block
            page = table[b][col] if col < len(table[b]) else -1
            if not 0 <= page < pages:
                status |= 1
                page = None
            entries = by_page.setdefault(col, (page, off, []))[2]
            if not live:
                status |= 1
                continue
            c, s = cos_sin[positions[t], :half], cos_sin[positions[t], half:]
            q_out[t] = to_bf16(rotate(bf16(q[t]), c, s, interleaved))
            key = rotate(bf16(k[t]), c, s, interleaved)
            k_out[t] = to_bf16(key)
            entries.append((off, key, bf16(v[t]).astype(np.float32)))
        for page, held, entries in by_page.values():
            if page is None:
                continue
            for side in (0, 1):
                for h in range(cache.heads):
                    new = [e[1 + side][h] for e in entries]
                    amax = max([np.nanmax(np.abs(x), initial=0.0) for x in new], default=0.0)
                    e = exponent(amax)
                    if held > 0:
                        old = int(np.clip(int(cache.scales[page, side, h]) - BIAS, LEAST, MOST))
                        if e > old:
                            rows = cache.codes[page, side, :held, h]
                            cache.codes[page, side, :held, h] = to_e4m3(
                                (e4m3(rows) * 2.0 ** (old - e)).astype(np.float32))
                        e = max(e, old)
                    cache.scales[page, side, h] = e + BIAS
                    for (off, _, _), x in zip(entries, new):
                        cache.codes[page, side, off, h] = to_e4m3(x.astype(np.float32) * np.float32(2.0 ** -e))
    return status


def attend(x, K, V, see, scale, weight_eps, tiny, q_lost=2.0 ** -39):
    """out, lse and tolerances of query rows x [R, D] over keys K, V [L, D] with see [R, L], in 64 bits.

    The kernels' arithmetic: the score error e_s is that of an fp32 sum of D
    exact products and of two more roundings, and of what the query's f16
    form loses (q_lost of its row's largest value; 0 where it stays bf16); a
    weight carries one rounding (weight_eps) and the exponential's 2^-20; a
    weight too small for its format's normal range is off by at most tiny [D]
    of the sum's unit, for each key; the two fp32 sums over n keys n 2^-24
    each; the result one bf16 rounding."""
    R, D = x.shape
    out, lse = np.zeros((R, V.shape[1])), np.full(R, -np.inf)
    tol_o, tol_l = np.zeros((R, V.shape[1])), np.zeros(R)
    for r in range(R):
        k, v = K[see[r]], V[see[r]]
        if not len(k):
            continue
        s = (k @ x[r]) * scale
        m = s.max()
        w = np.exp(s - m)
        den = w.sum()
        out[r] = (w @ v) / den
        lse[r] = m + np.log(den)
        size = abs(scale) * (np.abs(k) @ np.abs(x[r])).max()
        e_s = (D + 4) * 2.0 ** -24 * size + abs(scale) * np.abs(k).sum(1).max() * np.abs(x[r]).max() * q_lost
        sums = (len(k) + 32) * 2.0 ** -24
        tol_o[r] = (weight_eps + 2 * e_s + 2 * sums + 2.0 ** -18) * (w @ np.abs(v)) / den + len(k) * tiny \
            + 2.0 ** -8 * np.abs(out[r]) + 1e-30
        tol_l[r] = e_s + sums + 2.0 ** -19 + 2.0 ** -21 * abs(lse[r])
    return out, lse, tol_o, tol_l


def visible(n, length, first, window, sinks):
    """[n, length]: which keys the n queries at positions first, first + 1, ... see."""
    p, j = first + np.arange(n)[:, None], np.arange(length)[None]
    return (j <= p) & ((window <= 0) | (j > p - window) | (j < sinks))


def cached_attention(cache, q, start, lens, table, scale, window=0, sinks=0, gathered=False):
    """Attention over the cache.  Weights are f16 (2^-11), in units in which
    the largest is at least 2^6; what is below f16's normal range is off by
    2^-25 of them, times the reference scale, at most 2^6 above the largest of
    a value's page.  In calls of many rows per request and key head, and over
    gathered entries, they are bf16 (2^-8), queries stay bf16, and nothing else
    is rounded before the sums."""
    T, H, D = q.shape
    g = H // cache.heads
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    tol_o, tol_l = np.zeros((T, H, D)), np.zeros((T, H))
    pages = cache.codes.shape[0]
    gathered = gathered or max(np.diff(start), default=0) * g > {64: 48, 128: 32, 256: 24}[D]
    for b, length in enumerate(lens):
        t0, t1 = start[b], start[b + 1]
        n, length = t1 - t0, max(0, length)
        at = np.arange(length)
        col = at // cache.block
        page = np.where(col < len(table[b]), np.asarray(table[b])[np.minimum(col, len(table[b]) - 1)], -1)
        there = (page >= 0) & (page < pages)
        page = np.where(there, page, 0)
        see = np.repeat(visible(n, length, length - n, window, sinks) & there, g, 0)
        for kh in range(cache.heads):
            e = np.clip(cache.scales[page, :, kh].astype(int) - BIAS, LEAST, MOST)
            code = cache.codes[page, :, at % cache.block, kh]
            K, V = (e4m3(code[:, i]) * 2.0 ** e[:, i, None] for i in (0, 1))
            tiny = (2.0 ** -100 if gathered else 2.0 ** -25) * (2.0 ** e[:, 1].max() if length else 0.0) * 448
            rows = q[t0:t1, kh * g:(kh + 1) * g].reshape(n * g, D)
            got = attend(rows, K, V, see, scale, *((2.0 ** -8, tiny, 0.0) if gathered else (2.0 ** -11, tiny)))
            for to, x in zip((out, lse, tol_o, tol_l), got):
                to[t0:t1, kh * g:(kh + 1) * g] = x.reshape(n, g, *x.shape[1:])
    return out, lse, tol_o, tol_l


def prompt_attention(q, k, v, start, scale, window=0, sinks=0):
    """Attention over whole prompts.  Weights are bf16 (2^-8), flushed below 2^-126 of the largest."""
    T, H, D = q.shape
    KH = k.shape[1]
    g = H // KH
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    tol_o, tol_l = np.zeros((T, H, D)), np.zeros((T, H))
    for t0, t1 in zip(start[:-1], start[1:]):
        n = t1 - t0
        see = np.repeat(visible(n, n, 0, window, sinks), g, 0)
        for kh in range(KH):
            V = v[t0:t1, kh]
            rows = q[t0:t1, kh * g:(kh + 1) * g].reshape(n * g, D)
            got = attend(rows, k[t0:t1, kh], V, see, scale, 2.0 ** -8, 2.0 ** -100 * np.abs(V).max(initial=0), 0.0)
            for to, x in zip((out, lse, tol_o, tol_l), got):
                to[t0:t1, kh * g:(kh + 1) * g] = x.reshape(n, g, *x.shape[1:])
    return out, lse, tol_o, tol_l
