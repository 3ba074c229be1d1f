"""Serving from the per-head NVFP4 cache on the GPU: norm + rotation, window
and tree attention and the compaction of accepted drafts, each against the
plain 64-bit references (tolerances derived there from the arithmetic; bytes
compared whole)."""
import numpy as np
import pytest
import torch

import per_head_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
CANARY = 0x7B5A                                # bf16 pattern of rows that must stay as they were


@pytest.fixture(scope="module")
def kvq():
    from fp8_quantized_paged_concat_gb300 import _build
    _build.build()
    import fp8_quantized_paged_concat_gb300 as m
    m.load_library()
    return m


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def bf16_dev(bits):
    return dev(bits.view(np.int16)).view(torch.bfloat16)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def through_workspace(kvq, call, splits):
    """The arguments of a call whose ranges join through a workspace, not in clusters."""
    T, H, D = call["q"].shape
    need = max(16, kvq.kvq_per_head_attention_workspace_bytes(T, H, D, splits))
    return dict(call, num_splits=splits, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))


class Batch:
    """Requests with (context, new tokens), a shuffled block table, queries."""

    def __init__(self, reqs, heads, kv_heads, dim, block, layout, seed, extra_tokens=0, q_scale=1.0, pages=None):
        rng = np.random.default_rng(seed)
        self.reqs, self.rng = reqs, rng
        self.lens = [c + n for c, n in reqs]
        self.start = np.cumsum([0] + [n for _, n in reqs]).tolist()
        need = [max(1, -(-t // block)) for t in self.lens]
        total = sum(need) + 3
        order = rng.permutation(total)
        self.table = np.full((len(reqs), max(need) + 1), -1, np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = ref.Cache(1, total, block, kv_heads, dim, layout, rng)
        T = self.start[-1] + extra_tokens
        self.q_bits = ref.to_bf16(rng.standard_normal((T, heads, dim)) * q_scale)
        self.layout = layout
        self.k_scale, self.v_scale = np.float32(0.7), np.float32(1.3)
        self.scale = dim ** -0.5

    def device(self):
        return dict(q=bf16_dev(self.q_bits), query_start=i32(self.start), seq_lens=i32(self.lens),
                    block_table=i32(self.table.tolist()), kv_cache=dev(self.cache.raw[0]).view(self.cache.shape()[1:]),
                    k_scale=torch.tensor([self.k_scale], device=DEV), v_scale=torch.tensor([self.v_scale], device=DEV),
                    softmax_scale=self.scale, max_query_len=max([n for _, n in self.reqs] + [0]),
                    max_seq_len=max(self.lens + [0]), layout=self.layout)

    def want(self, **mask):
        return ref.attention(self.cache, ref.bf16(self.q_bits), self.start, self.lens, self.table, float(self.k_scale),
                             float(self.v_scale), self.scale, **mask)


def check(got, want, rows=None):
    out, lse, tol_o, tol_l = want
    o = ref.bf16(bits_of(got[0]))
    l = got[1].cpu().numpy().astype(np.float64)
    sl = slice(0, rows)
    err = np.abs(o[sl] - out[sl])
    assert np.all(err <= tol_o[sl]), f"out: worst error / tolerance {np.nanmax(err / tol_o[sl])}"
    dead = np.isneginf(lse[sl])
    assert np.array_equal(np.isneginf(l[sl]), dead)
    le = np.abs(l[sl][~dead] - lse[sl][~dead])
    assert np.all(le <= tol_l[sl][~dead]), f"lse: worst error / tolerance {np.max(le / tol_l[sl][~dead])}"


def random_tree(reqs, words, rng, empty=()):
    rows = []
    for _, n in reqs:
        seen = []
        for i in range(n):
            par = int(rng.integers(max(-1, i - 6), i))
            seen.append((1 << i) | (seen[par] if par >= 0 else 0))
        rows += [[(m >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for m in seen]
    for t in empty:
        rows[t] = [0] * words
    return rows


def mask_dev(rows):
    return dev(np.array(rows, np.uint64).reshape(len(rows), -1).view(np.int64))


# --------------------------------------------------------------------------
# window attention
# --------------------------------------------------------------------------

SHAPES = [(64, "NHD", 4, 4, 16), (64, "HND", 6, 2, 24), (128, "NHD", 8, 2, 16), (128, "HND", 7, 1, 16),
          (128, "NHD", 32, 2, 64), (256, "NHD", 4, 2, 16), (256, "HND", 10, 1, 8)]


@pytest.mark.parametrize("dim,layout,heads,kv,block", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (37, 4), (64, 40), (500, 1000)])
@pytest.mark.parametrize("splits", [1, 3, -3])
def test_window_decode(kvq, dim, layout, heads, kv, block, window, sinks, splits):
    """One new token per request: sequences of 1 (the token alone) up to
    several tiles, windows and sinks that cut inside pages and tiles."""
    b = Batch([(0, 1), (1, 1), (31, 1), (32, 1), (95, 1), (130, 1), (301, 1)], heads, kv, dim, block, layout, 11)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = dict(b.device(), num_splits=splits) if splits > 0 else through_workspace(kvq, b.device(), -splits)
    got = kvq.kvq_window_attention_nvfp4_per_head(**call, window=window, num_sinks=sinks, status=status)
    assert int(status.item()) == 0
    check(got, b.want(window=window, sinks=sinks))


@pytest.mark.parametrize("dim,layout,heads,kv,block", SHAPES)
@pytest.mark.parametrize("window,sinks,splits", [(0, 0, 1), (0, 0, 4), (0, 0, -2), (29, 5, 1), (29, 5, 2), (29, 5, -3),
                                                 (100, 0, 1), (0, 0, 8)])
def test_window_chunks(kvq, dim, layout, heads, kv, block, window, sinks, splits):
    """Chunks of new tokens: alone, behind a context, ragged, and none at all."""
    b = Batch([(0, 37), (50, 3), (17, 0), (120, 41), (0, 1), (70, 20)], heads, kv, dim, block, layout, 12)
    call = dict(b.device(), num_splits=splits) if splits > 0 else through_workspace(kvq, b.device(), -splits)
    got = kvq.kvq_window_attention_nvfp4_per_head(**call, window=window, num_sinks=sinks)
    check(got, b.want(window=window, sinks=sinks))


@pytest.mark.parametrize("new", [1, 130])
@pytest.mark.parametrize("splits", [1, 5, -5])
def test_padded_requests_see_nothing_and_other_rows_are_left(kvq, new, splits):
    """A padded request (length 0, or shorter than its query tokens) gives
    zeros and -inf where it sees nothing; rows behind the last request keep
    their contents, with and without an lse output."""
    b = Batch([(60, new), (0, new), (5, new)], 8, 2, 128, 16, "NHD", 13, extra_tokens=4)
    b.lens = [60 + new, 0, max(new - 3, 0)]
    d = dict(b.device(), num_splits=splits) if splits > 0 else through_workspace(kvq, b.device(), -splits)
    T = b.q_bits.shape[0]
    for with_lse in (True, False):
        out = torch.full((T, 8, 128), CANARY, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        lse = torch.full((T, 8), 123.0, device=DEV) if with_lse else False
        got = kvq.kvq_window_attention_nvfp4_per_head(**d, out=out, lse=lse)
        want = b.want()
        if with_lse:
            check(got, want, rows=T - 4)
            assert torch.all(got[1][T - 4:] == 123.0)
        else:
            assert got[1] is None
            assert np.all(np.abs(ref.bf16(bits_of(out))[:T - 4] - want[0][:T - 4]) <= want[2][:T - 4])
        assert np.all(bits_of(out)[T - 4:] == CANARY)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("splits", [1, 4])
def test_hidden_entries_have_no_effect(kvq, dim, new, splits):
    """NaN scales behind the sequences' ends, in the pages of no request, and
    in every entry that no query sees."""
    b = Batch([(200, new), (90, new)], 4, 2, dim, 16, "NHD", 14)
    window, sinks = 33, 3
    seen = set()
    for r, (ctx, n) in enumerate(b.reqs):
        for p in range(ctx + n):
            if p < sinks or p > ctx - window:
                seen.add((int(b.table[r, p // 16]), p % 16))
    for page in range(b.cache.raw.shape[1]):
        for off in range(16):
            if (page, off) not in seen:
                for h in range(2):
                    b.cache.raw[0, page, :, b.cache.spans(off, h)[1]] = 0x7F if (off + h) % 2 else 0xFF
    got = kvq.kvq_window_attention_nvfp4_per_head(**b.device(), window=window, num_sinks=sinks, num_splits=splits)
    check(got, b.want(window=window, sinks=sinks))


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("splits", [1, 4])
def test_later_tokens_nan_does_not_reach_earlier_rows(kvq, new, splits):
    """The last position's entry is NaN in keys and values: with several new
    tokens only the last row sees it (keys: NaN), the others are unaffected."""
    b = Batch([(100, new)], 4, 1, 128, 16, "HND", 15)
    p = b.lens[0] - 1
    b.cache.raw[0, b.table[0, p // 16], 1, b.cache.spans(p % 16, 0)[1]] = 0x7F
    if new > 1:
        b.cache.raw[0, b.table[0, p // 16], 0, b.cache.spans(p % 16, 0)[1]] = 0x7F
    got = kvq.kvq_window_attention_nvfp4_per_head(**b.device(), num_splits=splits)
    if new > 1:
        assert torch.isnan(got[0][-1]).all() and torch.isnan(got[1][-1]).all()
        b.cache.raw[0, b.table[0, p // 16], 0, b.cache.spans(p % 16, 0)[1]] = 0x30
        check(got, b.want(), rows=new - 1)
    else:
        check(got, b.want())


@pytest.mark.parametrize("new", [1, 40])
def test_bad_pages_and_requests(kvq, new):
    """Out-of-range pages and columns are skipped with a status bit; a request
    with a bad query range is left alone with another."""
    b = Batch([(100, new), (100, new), (100, new)], 4, 2, 128, 16, "NHD", 16)
    b.table[0, 2] = b.cache.raw.shape[1]
    b.table[1, 0] = -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = kvq.kvq_window_attention_nvfp4_per_head(**b.device(), status=status)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX
    check(got, b.want())
    # the table too narrow for the sequences
    status.zero_()
    full = b.table
    b.table = full[:, :4]
    got = kvq.kvq_window_attention_nvfp4_per_head(**b.device(), status=status)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX
    check(got, b.want())
    b.table = full
    # request 1's range is reversed
    d = b.device()
    for splits in (1, 3, 9):
        out = torch.full((3 * new, 4, 128), CANARY, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        status.zero_()
        bad = dict(d, query_start=i32([0, 2 * new, new, 3 * new]), seq_lens=i32([100 + new, 50, 100 + 2 * new]),
                   max_query_len=2 * new)
        kvq.kvq_window_attention_nvfp4_per_head(**bad, status=status, out=out, num_splits=splits)
        assert int(status.item()) & kvq.STATUS_BAD_BATCH
        status.zero_()
        out.view(torch.int16).fill_(CANARY)
        long = dict(d, max_query_len=new - 1)      # every request is longer than that
        kvq.kvq_window_attention_nvfp4_per_head(**long, status=status, out=out, num_splits=splits)
        if new > 1:
            assert int(status.item()) & kvq.STATUS_BAD_BATCH
        assert np.all(bits_of(out) == CANARY)


@pytest.mark.parametrize("new", [2, 90])
def test_strides_and_extreme_queries(kvq, new):
    """q as a slice of a packed projection, a strided output, and query rows
    whose values span bf16's range (row maxima from 2^-100 to 2^60)."""
    b = Batch([(70, new), (33, new)], 6, 2, 128, 16, "NHD", 17)
    T = 2 * new
    x = ref.bf16(b.q_bits)
    x[0] *= 2.0 ** -100
    x[1] *= 2.0 ** 60
    x[2, 0] = 0.0
    x[3, :, ::2] *= 2.0 ** -20
    b.q_bits = ref.to_bf16(x)
    b.scale = 2.0 ** -64 if new == 2 else 128 ** -0.5
    d = b.device()
    packed = torch.full((T, 10 * 128 + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    packed[:, 8:8 + 6 * 128] = d["q"].view(T, -1)
    d["q"] = packed[:, 8:8 + 6 * 128].view(T, 6, 128)
    out = torch.full((T, 7, 136), CANARY, dtype=torch.int16, device=DEV)
    o = out.view(torch.bfloat16)[:, :6, :128]
    got = kvq.kvq_window_attention_nvfp4_per_head(**d, out=o)
    assert got[0] is o
    if new == 2:
        check(got, b.want())
    else:
        want = b.want()
        keep = [t for t in range(T) if t != 1]       # 2^60: one key takes all the weight, and ties are not resolved
        check((got[0][keep], got[1][keep]), tuple(w[keep] for w in want))
    assert np.all(out[:, 6].cpu().numpy().view(np.uint16) == CANARY)
    assert np.all(out[:, :, 128:].cpu().numpy().view(np.uint16) == CANARY)


@pytest.mark.parametrize("new", [1, 50])
def test_scale_signs(kvq, new):
    """Scales of zero and below it: uniform weights over the visible keys, and the order of the scores reversed."""
    for scale in (0.0, -0.11):
        b = Batch([(75, new), (40, new)], 8, 2, 128, 16, "NHD", 20)
        b.scale = scale
        check(kvq.kvq_window_attention_nvfp4_per_head(**b.device(), window=40, num_sinks=3), b.want(window=40, sinks=3))


@pytest.mark.parametrize("new", [1, 64])
def test_offsets_past_32_bits(kvq, new):
    """Pages more than 2^32 bytes into the cache."""
    b = Batch([(150, new)], 8, 2, 128, 16, "NHD", 18)
    d = b.device()
    small = d["kv_cache"]
    page_bytes = small[0].numel()
    pages = (1 << 32) // page_bytes + 64
    big = torch.empty((pages, *small.shape[1:]), dtype=torch.uint8, device=DEV)
    n = small.shape[0]
    big[pages - n:] = small
    d.update(kv_cache=big, block_table=d["block_table"] + (pages - n))
    check(kvq.kvq_window_attention_nvfp4_per_head(**d), b.want())


def test_long_sequence_default_splits(kvq):
    """One request, 20000 positions: the default splits against one range, and both against the reference on a
    window that the reference can hold."""
    b = Batch([(20000, 1)], 8, 1, 128, 16, "NHD", 19)
    d = b.device()
    splits, use_workspace = kvq.kvq_per_head_attention_default_splits(1, 8, 1, 128, 1, 20001)
    assert splits > kvq.PER_HEAD_CLUSTER_SPLITS and use_workspace
    a0, l0 = kvq.kvq_window_attention_nvfp4_per_head(**d)
    a1, l1 = kvq.kvq_window_attention_nvfp4_per_head(**d, num_splits=1)
    want = b.want()
    check((a0, l0), want)
    check((a1, l1), want)
    # a max_seq_len that is too small only makes the ranges uneven
    a2, l2 = kvq.kvq_window_attention_nvfp4_per_head(**through_workspace(kvq, dict(d, max_seq_len=64), 7))
    check((a2, l2), want)
    check(kvq.kvq_window_attention_nvfp4_per_head(**d, num_splits=8), want)


# --------------------------------------------------------------------------
# tree attention
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dim,layout,heads,kv,block", SHAPES)
@pytest.mark.parametrize("splits", [1, 3, -4])
def test_tree(kvq, dim, layout, heads, kv, block, splits):
    """Random trees behind contexts of 0 to several tiles, up to 70 drafts
    (two mask words), masks that leave a draft nothing but the context and,
    without a context, nothing at all."""
    b = Batch([(0, 5), (1, 1), (100, 70), (64, 64), (33, 17), (0, 3)], heads, kv, dim, block, layout, 21)
    rows = random_tree(b.reqs, 2, b.rng, empty=(2, 7, 157))
    call = dict(b.device(), num_splits=splits) if splits > 0 else through_workspace(kvq, b.device(), -splits)
    got = kvq.kvq_tree_attention_nvfp4_per_head(**call, tree_mask=mask_dev(rows))
    want = b.want(tree=rows)
    assert np.isneginf(want[1][2]).all() and np.isneginf(want[1][157]).all()
    check(got, want)


def test_tree_chain_equals_causal_window(kvq):
    """A tree that is one chain is plain causal attention: bit for bit the
    window form without a window."""
    b = Batch([(77, 40), (10, 33)], 8, 2, 128, 16, "NHD", 22)
    rows = [[(2 << i) - 1] for _, n in b.reqs for i in range(n)]
    d = b.device()
    to, tl = kvq.kvq_tree_attention_nvfp4_per_head(**d, tree_mask=mask_dev(rows), num_splits=1)
    check((to, tl), b.want())


def test_tree_garbage_bits_and_wide_masks(kvq):
    """Bits past a request's drafts are ignored; mask rows may be slices of
    wider ones."""
    b = Batch([(40, 9), (20, 12)], 4, 2, 64, 16, "HND", 23)
    rows = random_tree(b.reqs, 1, b.rng)
    dirty, t = [], 0
    for _, n in b.reqs:
        for _ in range(n):
            dirty.append([rows[t][0] | ((2 ** 64 - 1) & ~((1 << n) - 1)), 2 ** 64 - 1, 2 ** 64 - 1])
            t += 1
    mask = mask_dev(dirty)[:, :1]
    assert mask.stride(0) == 3
    check(kvq.kvq_tree_attention_nvfp4_per_head(**b.device(), tree_mask=mask), b.want(tree=rows))


# --------------------------------------------------------------------------
# norm and rotation
# --------------------------------------------------------------------------

@pytest.mark.parametrize("heads,kv,dim,rot", [(8, 2, 128, 128), (5, 3, 64, 64), (16, 1, 256, 64), (3, 1, 80, 80),
                                              (4, 4, 96, 32), (2, 2, 16, 16), (7, 1, 128, 0), (40, 8, 128, 64)])
@pytest.mark.parametrize("tokens", [1, 37, 1500])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(kvq, heads, kv, dim, rot, tokens, interleaved):
    rng = np.random.default_rng(31)
    width = (heads + 2 * kv) * dim
    qkv = ref.to_bf16(rng.standard_normal((tokens, width)) * 3)
    qkv[0, :dim] = 0                                             # a head of zeros
    wq, wk = (ref.to_bf16(1 + 0.3 * rng.standard_normal(dim)) for _ in range(2))
    max_pos = 500
    pos = rng.integers(0, max_pos, tokens)
    pos[0] = max_pos - 1
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32).reshape(max_pos, rot)
    x = bf16_dev(qkv)
    q, k = x[:, :heads * dim].view(tokens, heads, dim), x[:, heads * dim:-kv * dim].view(tokens, kv, dim)
    args = (bf16_dev(wq), bf16_dev(wk), dev(pos), dev(table), 1e-6)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo, ko = kvq.kvq_qk_norm_rope(q, k, *args, interleaved=interleaved, status=status)
    assert int(status.item()) == 0
    for got, src, w in ((qo, q, wq), (ko, k, wk)):
        want, tol = ref.norm_rope(ref.bf16(bits_of(src)), ref.bf16(w), pos, table, rot, 1e-6, interleaved)
        err = np.abs(ref.bf16(bits_of(got)) - want)
        assert np.all(err <= tol), f"worst error / tolerance {np.max(err / tol)}"
    # in place, in the packed rows, gives the same bits and leaves the values alone
    kvq.kvq_qk_norm_rope(q, k, *args, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q.contiguous().view(torch.int16), qo.view(torch.int16))
    assert torch.equal(k.contiguous().view(torch.int16), ko.view(torch.int16))
    assert np.array_equal(bits_of(x)[:, -kv * dim:], qkv[:, -kv * dim:])


def test_norm_rope_bad_positions_are_skipped(kvq):
    rng = np.random.default_rng(32)
    q = bf16_dev(ref.to_bf16(rng.standard_normal((6, 4, 64))))
    k = bf16_dev(ref.to_bf16(rng.standard_normal((6, 2, 64))))
    w = bf16_dev(ref.to_bf16(np.ones(64)))
    table = dev(rng.standard_normal((10, 64)).astype(np.float32))
    pos = dev(np.array([0, 10, 9, -1, 2 ** 40, 3]))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = [torch.full(t.shape, CANARY, dtype=torch.int16, device=DEV).view(torch.bfloat16) for t in (q, k)]
    kvq.kvq_qk_norm_rope(q, k, w, w, pos, table, 1e-5, q_out=outs[0], k_out=outs[1], status=status)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX
    for o in outs:
        got = bits_of(o).reshape(6, -1)
        assert np.all(got[[1, 3, 4]] == CANARY) and not np.any(np.all(got[[0, 2, 5]] == CANARY, axis=1))


# --------------------------------------------------------------------------
# compaction
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dim,layout,kv,block", [(128, "NHD", 2, 16), (128, "HND", 3, 16), (64, "NHD", 4, 24),
                                                 (256, "HND", 1, 8), (80, "NHD", 2, 16), (16, "HND", 2, 8),
                                                 (96, "HND", 1, 16)])
@pytest.mark.parametrize("layers", [1, 3])
def test_compact(kvq, dim, layout, kv, block, layers):
    """Accepted lists from none to all, chains that overlap their own
    destinations, and long ones that take several chunks."""
    b = Batch([(0, 5), (13, 40), (31, 16), (7, 1), (50, 300), (20, 64)], kv, kv, dim, block, layout, 41)
    rng = np.random.default_rng(42)
    b.cache = ref.Cache(layers, b.cache.raw.shape[1], block, kv, dim, layout, rng)
    acc = np.full((6, 290), -7, np.int32)
    lists = [[4], list(range(1, 40)), [], [0], sorted(rng.choice(300, 290, replace=False)), [0, 1, 5, 63]]
    for r, a in enumerate(lists):
        acc[r, :len(a)] = a
    lens = [len(a) for a in lists]
    cache = dev(b.cache.raw).view(b.cache.shape())
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kvq.kvq_compact_drafts_nvfp4_per_head(cache if layers > 1 else cache[0], i32(b.start), i32(b.lens), dev(acc),
                                          i32(lens), i32(b.table.tolist()), layout=layout, status=status)
    want = ref.compact(b.cache, b.start, b.lens, acc, lens, b.table)
    assert int(status.item()) == 0
    assert np.array_equal(cache.cpu().numpy().reshape(want.shape), want)
    assert not np.array_equal(want, b.cache.raw)


def test_compact_malformed_lists_leave_the_request(kvq):
    b = Batch([(20, 8)] * 7, 2, 2, 64, 16, "NHD", 43)
    acc = np.array([[1, 1, 2], [2, 1, 3], [0, 1, 8], [-1, 0, 1], [1, 2, 3], [3, 5, 7], [1, 3, 5]], np.int32)
    lens = [3, 3, 3, 3, 4, -1, 3]
    b.lens[6] = 5                                           # shorter than its drafts
    cache = dev(b.cache.raw[0]).view(b.cache.shape()[1:])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kvq.kvq_compact_drafts_nvfp4_per_head(cache, i32(b.start), i32(b.lens), dev(acc), i32(lens), i32(b.table.tolist()),
                                          status=status)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX | kvq.STATUS_BAD_BATCH
    assert np.array_equal(cache.cpu().numpy().reshape(b.cache.raw[0].shape), b.cache.raw[0])
    # bad pages: those moves alone are skipped
    b = Batch([(20, 8)], 2, 2, 64, 4, "NHD", 44)
    b.table[0, 6] = 10 ** 6
    acc, status = np.array([[1, 5, 7]], np.int32), torch.zeros(1, dtype=torch.int32, device=DEV)
    cache = dev(b.cache.raw[0]).view(b.cache.shape()[1:])
    kvq.kvq_compact_drafts_nvfp4_per_head(cache, i32(b.start), i32(b.lens), dev(acc), i32([3]), i32(b.table.tolist()),
                                          status=status)
    want = ref.compact(b.cache, b.start, b.lens, acc, [3], b.table)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX
    assert np.array_equal(cache.cpu().numpy().reshape(want[0].shape), want[0])


# --------------------------------------------------------------------------
# together, in graphs and on streams
# --------------------------------------------------------------------------

def test_speculative_step_end_to_end(kvq):
    """A draft step as an engine runs it: normalise and rotate, write the
    drafts' keys and values, tree attention, accept a path, compact, then a
    decode step whose result equals that of a cache which only ever held the
    accepted tokens."""
    rng = np.random.default_rng(51)
    H, KH, D, block, ctx, n = 8, 2, 128, 16, 37, 12
    path = [1, 4, 9]
    ang = np.arange(128)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
    table_cs = dev(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    w = bf16_dev(ref.to_bf16(1 + 0.1 * rng.standard_normal(D)))
    one = torch.ones(1, device=DEV)
    table = i32([[5, 2, 7, 1, 3]])
    slots = lambda pos: dev(np.array([[5, 2, 7, 1, 3][p // block] * block + p % block for p in pos]))  # noqa: E731

    def step(cache, x, pos, slot_pos, mask, length):
        t = len(pos)
        q, k, v = (x[:, a * D:b * D].view(t, b - a, D) for a, b in ((0, H), (H, H + KH), (H + KH, H + 2 * KH)))
        q, k = kvq.kvq_qk_norm_rope(q, k, w, w, dev(np.array(pos)), table_cs, 1e-6)
        kvq.kvq_reshape_and_cache_nvfp4(k, v, cache, slots(slot_pos), one, one)
        args = (one, one, D ** -0.5, t, length)
        if mask is None:
            return kvq.kvq_window_attention_nvfp4_per_head(q, i32([0, t]), i32([length]), table, cache, *args)
        return kvq.kvq_tree_attention_nvfp4_per_head(q, i32([0, t]), i32([length]), mask, table, cache, *args)

    def inputs(t):
        return bf16_dev(ref.to_bf16(rng.standard_normal((t, (H + 2 * KH) * D))))

    shape = (9, 2, block, KH, D // 2 + D // 16)
    a, b = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
    prompt, drafts, last = inputs(ctx), inputs(n), inputs(1)
    pa = step(a, prompt, list(range(ctx)), list(range(ctx)), None, ctx)
    step(b, prompt, list(range(ctx)), list(range(ctx)), None, ctx)
    assert torch.isfinite(pa[0]).all()
    # the tree: the path's drafts are each other's ancestors; the others hang off the context
    seen = [1 << i for i in range(n)]
    for u, v in zip(path, path[1:]):
        seen[v] |= seen[u]
    depth = [bin(m).count("1") for m in seen]
    tree = step(a, drafts, [ctx + d - 1 for d in depth], list(range(ctx, ctx + n)), mask_dev([[m] for m in seen]), ctx + n)
    chain = step(b, drafts[path].contiguous(), list(range(ctx, ctx + 3)), list(range(ctx, ctx + 3)), None, ctx + 3)
    # the path's rows see the same keys in the same order in both: equal but for the sums' grouping
    assert torch.allclose(tree[0][path].float(), chain[0].float(), rtol=2 ** -7, atol=2 ** -9)
    assert torch.allclose(tree[1][path], chain[1], atol=1e-5)
    kvq.kvq_compact_drafts_nvfp4_per_head(a, i32([0, n]), i32([ctx + n]), i32([path]), i32([3]), table)
    end = ctx + 3
    ra = step(a, last, [end], [end], None, end + 1)
    rb = step(b, last, [end], [end], None, end + 1)
    assert torch.equal(ra[0].view(torch.int16), rb[0].view(torch.int16)) and torch.equal(ra[1], rb[1])


@pytest.mark.parametrize("new,splits,joined", [(1, 4, "cluster"), (1, 4, "workspace"), (1, 1, "cluster"),
                                               (80, 1, "workspace"), (80, 2, "workspace")])
def test_graphs_and_streams(kvq, new, splits, joined):
    """Two captured calls with workspaces of their own, replayed on new
    inputs, and a call on a side stream give the eager call's bits."""
    bs = [Batch([(300, new), (40, new)], 8, 2, 128, 16, "NHD", 61 + i) for i in range(2)]
    ds = [b.device() for b in bs]
    cluster = joined == "cluster"
    eager = [kvq.kvq_window_attention_nvfp4_per_head(**(dict(d, num_splits=splits) if cluster else
                                                        through_workspace(kvq, d, splits))) for d in ds]
    need = kvq.kvq_per_head_attention_workspace_bytes(2 * new, 8, 128, splits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(eager[0][0])
    lse = torch.empty_like(eager[0][1])
    kvq.kvq_window_attention_nvfp4_per_head(**ds[0], num_splits=splits, out=out, lse=lse, stream=side,
                                            workspace=None if cluster else
                                            torch.empty(need, dtype=torch.uint8, device=DEV))
    side.synchronize()
    assert torch.equal(out.view(torch.int16), eager[0][0].view(torch.int16)) and torch.equal(lse, eager[0][1])
    graphs = []
    for i in range(2):
        d = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in ds[i].items()}
        ws = None if cluster else torch.empty(need, dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = kvq.kvq_window_attention_nvfp4_per_head(**d, num_splits=splits, workspace=ws)
        graphs.append((g, d, got, ws))
    for swap in (False, True):
        for i, (g, d, got, _) in enumerate(graphs):
            for k, v in ds[1 - i if swap else i].items():
                if isinstance(v, torch.Tensor) and v.shape == d[k].shape:
                    d[k].copy_(v)
            g.replay()
        torch.cuda.synchronize()
        for i, (_, _, got, _) in enumerate(graphs):
            want = eager[1 - i if swap else i]
            assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("raw", [False, True])
def test_side_stream_results_and_workspaces_are_the_streams(kvq, raw):
    """Calls on another stream that allocate their results and workspace: bits
    of the eager calls, whatever the current stream does with freed memory."""
    b = Batch([(900, 60), (333, 60)], 8, 2, 128, 16, "NHD", 71)
    d = b.device()
    eager = kvq.kvq_window_attention_nvfp4_per_head(**d, num_splits=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got.append(kvq.kvq_window_attention_nvfp4_per_head(**d, num_splits=4,
                                                           stream=side.cuda_stream if raw else side))
        # as large as the workspace just given back, and written at once on the current stream
        torch.empty(kvq.kvq_per_head_attention_workspace_bytes(120, 8, 128, 4), dtype=torch.uint8, device=DEV).fill_(0xFF)
    torch.cuda.current_stream().wait_stream(side)
    for out, lse in got:
        assert torch.equal(out.view(torch.int16), eager[0].view(torch.int16)) and torch.equal(lse, eager[1])


def test_shared_pages_and_the_widest_batch(kvq):
    """The largest batch, its requests all on the same pages with the same
    query: every row has the first one's bits, and those are right."""
    b = Batch([(33, 1)], 4, 2, 64, 16, "NHD", 72)
    d = b.device()
    n = 65535
    d.update(q=d["q"].expand(n, -1, -1), query_start=torch.arange(n + 1, dtype=torch.int32, device=DEV),
             seq_lens=d["seq_lens"].expand(n).contiguous(), block_table=d["block_table"].expand(n, -1).contiguous())
    for splits in (1, 2):
        out, lse = kvq.kvq_window_attention_nvfp4_per_head(**d, num_splits=splits)
        check((out[:1], lse[:1]), b.want())
        assert torch.equal(out.view(torch.int16), out[:1].view(torch.int16).expand_as(out))
        assert torch.equal(lse, lse[:1].expand_as(lse))


def test_python_calls_refuse_what_does_not_fit(kvq):
    """Types, shapes, layouts and workspaces that no launch may see."""
    b = Batch([(40, 1), (8, 1)], 4, 2, 128, 16, "NHD", 73)
    d = b.device()
    call = kvq.kvq_window_attention_nvfp4_per_head
    wrong = [("q", d["q"].float(), "q: expected"), ("q", d["q"][0], "q: expected"), ("q", d["q"][..., ::2], "q: expected"),
             ("query_start", d["query_start"][:-1], "query_start: expected"),
             ("seq_lens", d["seq_lens"].long(), "seq_lens: expected"), ("seq_lens", d["seq_lens"].cpu(), "seq_lens: expected"),
             ("block_table", d["block_table"][:1], "block_table: expected"),
             ("kv_cache", d["kv_cache"][:, :1], "kv_cache: expected"), ("kv_cache", d["kv_cache"][:, :, ::2], "kv_cache: expected"),
             ("kv_cache", d["kv_cache"][..., :-9], "kv_cache: expected"), ("layout", "NDH", "layout: expected"),
             ("layout", 1, "layout: expected"), ("k_scale", d["k_scale"].double(), "k_scale: expected"),
             ("max_query_len", 1 << 31, "max_query_len: out of range"),
             ("out", torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV), "out: expected"),
             ("lse", torch.empty(2, 3, device=DEV), "lse: expected"),
             ("status", torch.empty(0, dtype=torch.int32, device=DEV), "status: expected")]
    for name, value, needle in wrong:
        with pytest.raises(ValueError, match=needle):
            call(**{**d, name: value})
    with pytest.raises(RuntimeError, match="workspace must be"):
        call(**d, num_splits=2, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(RuntimeError, match="num_splits"):
        call(**d, num_splits=129)
    with pytest.raises(RuntimeError, match="head_size"):
        q = torch.zeros(2, 4, 96, dtype=torch.bfloat16, device=DEV)
        call(**dict(d, q=q, kv_cache=torch.zeros(4, 2, 16, 2, 54, dtype=torch.uint8, device=DEV)))
    with pytest.raises(ValueError, match="tree_mask: expected"):
        tree = {k: v for k, v in d.items()}
        kvq.kvq_tree_attention_nvfp4_per_head(**tree, tree_mask=torch.zeros(1, 1, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="accepted_lens: expected"):
        kvq.kvq_compact_drafts_nvfp4_per_head(d["kv_cache"], d["query_start"], d["seq_lens"], i32([[0], [0]]), i32([1]),
                                              d["block_table"])
    with pytest.raises(ValueError, match="positions: expected"):
        w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
        kvq.kvq_qk_norm_rope(d["q"], d["q"], w, w, i32([0, 1]), torch.zeros(8, 128, device=DEV), 1e-6)
    out, lse = call(**d)                                    # nothing above left an error behind
    check((out, lse), b.want())


@pytest.mark.parametrize("new,ctx", [(1, 9000), (24, 3000), (100, 5000)])
def test_calls_at_once_and_captured_with_default_ranges(kvq, new, ctx):
    """Two calls in flight on two streams, and a captured call that sizes its
    ranges and allocates its workspace itself, replayed: the eager bits."""
    bs = [Batch([(ctx, new)], 8, 2, 128, 16, "NHD", 81 + i) for i in range(2)]
    masks = [mask_dev(random_tree([(ctx, new)], 2, b.rng)) for b in bs]
    ds = [b.device() for b in bs]
    for d, m in zip(ds, masks):
        d["tree_mask"] = m
    eager = [kvq.kvq_tree_attention_nvfp4_per_head(**d) for d in ds]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[kvq.kvq_tree_attention_nvfp4_per_head(**d, stream=s) for d, s in zip(ds, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    d = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in ds[0].items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = kvq.kvq_tree_attention_nvfp4_per_head(**d)
    for i in (0, 1, 0):
        for k, v in ds[i].items():
            if isinstance(v, torch.Tensor):
                d[k].copy_(v)
        g.replay()
        torch.cuda.synchronize()
        got.append([tuple(t.clone() for t in captured) if j == i else eager[j] for j in range(2)])
    for pair in got:
        for (out, lse), want in zip(pair, eager):
            assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])


def test_compact_layers_apart_in_memory(kvq):
    """Layers that are slices of a larger allocation: what lies between them stays."""
    rng = np.random.default_rng(91)
    cache = ref.Cache(3, 6, 16, 2, 128, "NHD", rng)
    table = np.array([[3, 1, 5]])
    start, lens, acc, n = [0, 9], [40], np.array([[1, 4, 6, 8]]), [4]
    inner = cache.shape()[1:]
    whole = torch.full((3, 6 + 2, *inner[1:]), 0xA5, dtype=torch.uint8, device=DEV)
    view = whole[:, :6]
    view.copy_(dev(cache.raw).view(cache.shape()))
    kvq.kvq_compact_drafts_nvfp4_per_head(view, i32(start), i32(lens), i32(acc.tolist()), i32(n), i32(table.tolist()))
    want = ref.compact(cache, start, lens, acc, n, table)
    np.testing.assert_array_equal(view.reshape(want.shape).cpu().numpy(), want)
    assert torch.all(whole[:, 6:] == 0xA5)


@pytest.mark.parametrize("new", [1, 20])
def test_a_chain_of_calls_runs_in_order(kvq, new):
    """Each call reads what the one before it wrote (queries, cache entries,
    the in-place rotation): queued and captured, the bits of a run that waits
    after every call."""
    b = Batch([(700, new), (90, new), (33, new)], 8, 2, 128, 16, "NHD", 95)
    d = b.device()
    T = b.start[-1]
    w = bf16_dev(ref.to_bf16(1 + 0.1 * b.rng.standard_normal(128)))
    table = dev(b.rng.standard_normal((800, 128)).astype(np.float32))
    pos = dev(b.rng.integers(0, 800, T))
    accepted, count = i32([[new - 1]] * 3), i32([1] * 3)
    kept = {k: d[k].clone() for k in ("q", "kv_cache")}

    def chain(wait):
        q, cache = kept["q"].clone(), kept["kv_cache"].clone()
        k = q[:, :2].clone()
        out = []
        for _ in range(12):
            kvq.kvq_qk_norm_rope(q, k, w, w, pos, table, 1e-6, q_out=q, k_out=k)
            wait()
            kvq.kvq_compact_drafts_nvfp4_per_head(cache, d["query_start"], d["seq_lens"], accepted, count, d["block_table"])
            wait()
            o, lse = kvq.kvq_window_attention_nvfp4_per_head(**{**d, "q": q, "kv_cache": cache})
            wait()
            q, k = o, o[:, 2:4].clone()
            wait()
            out += [o.clone(), lse]
        return out + [cache]

    want = chain(torch.cuda.synchronize)
    got = [chain(lambda: None)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = chain(lambda: None)
    g.replay()
    torch.cuda.synchronize()
    for run in (*got, captured):
        for a, c in zip(run, want):
            assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def test_out_of_memory_is_torchs_own_error(kvq):
    """A workspace past the allocator's limit (set low for the call): torch's
    error, and the next call is as before."""
    b = Batch([(300, 1)], 8, 2, 128, 16, "NHD", 97)
    d = b.device()
    want = kvq.kvq_window_attention_nvfp4_per_head(**d)
    q = torch.zeros(1 << 16, 8, 128, dtype=torch.bfloat16, device=DEV)       # 128 MiB; 32 GiB of workspace
    wide = dict(d, q=q, query_start=i32([0, 1]), num_splits=128)
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.02)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            kvq.kvq_window_attention_nvfp4_per_head(**wide)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    got = kvq.kvq_window_attention_nvfp4_per_head(**d)
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("new", [1, 40])
def test_what_the_kernel_before_wrote_is_what_is_read(kvq, new):
    """Lengths, tables, masks, positions and scales written by a kernel that
    is queued directly before the call: the bits of a run that waits."""
    b = Batch([(400, new), (90, new)], 8, 2, 128, 16, "NHD", 98)
    d = b.device()
    d["tree_mask"] = mask_dev(random_tree(b.reqs, 1, b.rng))
    T = b.start[-1]
    w = bf16_dev(ref.to_bf16(1 + 0.1 * b.rng.standard_normal(128)))
    table = dev(b.rng.standard_normal((800, 128)).astype(np.float32))
    pos = dev(b.rng.integers(0, 800, T))
    names = ("seq_lens", "block_table", "tree_mask", "k_scale", "v_scale", "query_start")
    other = {n: d[n].clone() for n in names}
    other["seq_lens"] = d["seq_lens"] - i32([37, 11])
    other["block_table"] = d["block_table"].flip(0).contiguous()
    other["tree_mask"] = torch.zeros_like(d["tree_mask"])
    other["k_scale"], other["v_scale"] = d["k_scale"] * 0.5, d["v_scale"] * -2
    pos2, w2 = pos.flip(0).contiguous(), (w.float() * 0.5).bfloat16()

    def rounds(wait):
        live = {n: d[n].clone() for n in names}
        p, wl = pos.clone(), w.clone()
        out = []
        for i in range(8):
            for n in names:
                live[n].copy_((other if i % 2 else d)[n])
                wait()
            out += kvq.kvq_tree_attention_nvfp4_per_head(**{**d, **live})
            wait()
            wl.copy_(w2 if i % 2 else w)
            p.copy_(pos2 if i % 2 else pos)
            wait()
            out += kvq.kvq_qk_norm_rope(d["q"], d["q"], wl, wl, p, table, 1e-6)
            wait()
        return out

    want, got = rounds(torch.cuda.synchronize), rounds(lambda: None)
    assert all(torch.equal(a.view(torch.uint8), c.view(torch.uint8)) for a, c in zip(got, want))


@pytest.mark.parametrize("dim,heads,kv,new", [(64, 8, 2, 3), (64, 8, 2, 5), (64, 10, 2, 3), (128, 8, 2, 3), (128, 14, 2, 4)])
@pytest.mark.parametrize("tree", [False, True])
def test_many_requests_of_a_few_rows(kvq, dim, heads, kv, new, tree):
    """Enough requests to fill the GPU with blocks of 16 query rows (ragged
    lengths, 9 to 28 rows per request and key head)."""
    rng = np.random.default_rng(99)
    reqs = [(int(c), new if i % 3 else int(rng.integers(0, new + 1))) for i, c in enumerate(rng.integers(0, 50, 240))]
    b = Batch(reqs, heads, kv, dim, 16, "NHD", 100)
    d = dict(b.device(), max_query_len=new)
    if tree:
        rows = random_tree(reqs, 1, b.rng, empty=(3, 17))
        check(kvq.kvq_tree_attention_nvfp4_per_head(**d, tree_mask=mask_dev(rows)), b.want(tree=rows))
    else:
        check(kvq.kvq_window_attention_nvfp4_per_head(**d, window=21, num_sinks=2), b.want(window=21, sinks=2))
    check(kvq.kvq_window_attention_nvfp4_per_head(**through_workspace(kvq, d, 3)), b.want())


@pytest.mark.parametrize("dim,heads,kv,new", [(64, 6, 2, 11), (64, 6, 2, 21), (64, 6, 2, 22), (128, 8, 2, 8), (128, 8, 2, 9),
                                              (256, 4, 2, 8), (256, 4, 2, 9), (256, 4, 2, 16)])
@pytest.mark.parametrize("splits", [1, 2, -2, None])
def test_rows_on_both_sides_of_the_kernels_limits(kvq, dim, heads, kv, new, splits):
    """33 to 66 rows at head size 64, 32 and 36 at 128, 16 to 32 at 256: whole,
    in clusters where the call may, and through a workspace."""
    reqs = [(70, new), (3, new), (300, new - 1)]
    b = Batch(reqs, heads, kv, dim, 16, "HND", 101)
    d = b.device()
    rows = random_tree(reqs, 1, b.rng, empty=(1,))
    if splits is not None:
        d = through_workspace(kvq, d, -splits) if splits < 0 else dict(d, num_splits=splits)
    check(kvq.kvq_tree_attention_nvfp4_per_head(**d, tree_mask=mask_dev(rows)), b.want(tree=rows))
    check(kvq.kvq_window_attention_nvfp4_per_head(**d, window=100, num_sinks=5), b.want(window=100, sinks=5))


@pytest.mark.parametrize("new,splits", [(1, 4), (1, 40), (40, 3)])
def test_what_the_kernel_before_wrote_is_what_the_join_reads(kvq, new, splits):
    """The same for a call whose ranges join through a workspace, in a second
    kernel: lengths, query ranges and value scale written directly before it."""
    b = Batch([(900, new), (700, new), (90, new)], 8, 2, 128, 16, "NHD", 102)
    d = through_workspace(kvq, b.device(), splits)
    names = ("query_start", "seq_lens", "v_scale")
    other = dict(query_start=i32([0, new, new, 3 * new]), seq_lens=d["seq_lens"] - i32([37, 300, 5]),
                 v_scale=d["v_scale"] * -2)
    d["max_query_len"] = 2 * new

    def rounds(wait):
        live = {n: d[n].clone() for n in names}
        out = []
        for i in range(16):
            for n in names:
                live[n].copy_((other if i % 2 else d)[n])
                wait()
            o = torch.full((3 * new, 8, 128), CANARY, dtype=torch.int16, device=DEV).view(torch.bfloat16)
            wait()
            out += kvq.kvq_window_attention_nvfp4_per_head(**{**d, **live}, out=o)
            wait()
        return out

    want, got = rounds(torch.cuda.synchronize), rounds(lambda: None)
    assert all(torch.equal(a.view(torch.uint8), c.view(torch.uint8)) for a, c in zip(got, want))
    check(want[:2], b.want())
    b.start, b.lens, b.v_scale = [0, new, new, 3 * new], other["seq_lens"].tolist(), b.v_scale * np.float32(-2)
    check(want[2:4], b.want())


def test_a_workspace_that_the_default_ranges_do_not_need(kvq):
    """An engine keeps one workspace for all its calls: a call whose default
    ranges join in a cluster runs as without it, however small it is, and one
    whose ranges need it uses it."""
    b = Batch([(2000, 1)], 8, 2, 128, 16, "NHD", 103)
    d = b.device()
    splits, use_workspace = kvq.kvq_per_head_attention_default_splits(1, 8, 2, 128, 1, 2001)
    assert splits > 1 and not use_workspace
    want = kvq.kvq_window_attention_nvfp4_per_head(**d)
    check(want, b.want())
    mine = torch.full((64,), 0x5A, dtype=torch.uint8, device=DEV)
    got = kvq.kvq_window_attention_nvfp4_per_head(**d, workspace=mine)
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])
    assert torch.all(mine == 0x5A)
    with pytest.raises(ValueError, match="workspace: expected"):
        kvq.kvq_window_attention_nvfp4_per_head(**d, workspace=mine.cpu())
    # ranges asked for by number go through the workspace that is given
    with pytest.raises(RuntimeError, match="workspace must be"):
        kvq.kvq_window_attention_nvfp4_per_head(**d, workspace=mine, num_splits=splits)
    b = Batch([(20000, 1)], 8, 1, 128, 16, "NHD", 104)
    d = b.device()
    splits, use_workspace = kvq.kvq_per_head_attention_default_splits(1, 8, 1, 128, 1, 20001)
    assert use_workspace
    with pytest.raises(RuntimeError, match="workspace must be"):
        kvq.kvq_window_attention_nvfp4_per_head(**d, workspace=mine)
    mine = torch.zeros(kvq.kvq_per_head_attention_workspace_bytes(1, 8, 128, splits), dtype=torch.uint8, device=DEV)
    got, want = kvq.kvq_window_attention_nvfp4_per_head(**d, workspace=mine), kvq.kvq_window_attention_nvfp4_per_head(**d)
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.any(mine != 0)


# --------------------------------------------------------------------------
# a running maximum that grows
# --------------------------------------------------------------------------

GROWTH_SIGNS = (1.0, 1.0, 0.4, -1.0)           # of a key head's four query heads: two grow, one slowly, one falls


def growing_batch(reqs, dim, layout, seed, unit, per_step):
    """Four query heads on one key head whose scores rise with the position:
    a key of 32-key step i has ones in per_step * i of its dimensions (each
    worth `unit` in base two to the first two heads) and zeros elsewhere."""
    b = Batch(reqs, 4, 1, dim, 16, layout, seed)
    for r, length in enumerate(b.lens):
        for p in range(length):
            page, off = b.table[r, p // 16], p % 16
            code = np.zeros(dim, np.uint8)
            code[b.rng.permutation(dim)[:per_step * (p // 32)]] = 2              # e2m1 1.0
            data, scales = b.cache.spans(off, 0)
            b.cache.raw[0, page, 0, data] = code[0::2] | code[1::2] << 4
            b.cache.raw[0, page, 0, scales] = 0x38                               # e4m3 1.0
    c = unit / (np.log2(np.e) * b.scale * float(b.k_scale))
    q = c * np.array(GROWTH_SIGNS)[None, :, None] * (1 + 0.05 * b.rng.standard_normal(b.q_bits.shape))
    b.q_bits = ref.to_bf16(q)
    return b


def base_two_scores(b, token, head):
    """The row's scores of the first request's keys up to its own position."""
    ctx = b.reqs[0][0]
    keys = np.stack([k for k, _ in ref.keys_of(b.cache, b.table[0], 0, range(ctx + token + 1))])
    return (keys @ ref.bf16(b.q_bits)[token, head]) * (np.log2(np.e) * b.scale * float(b.k_scale))


def growths(scores, steps):
    """How often a reference maximum, taken from the first of `steps` (lists
    of groups of keys), is exceeded by a group whose weights against it sum to
    more than 2^8, each time taking the step's maximum; and the last such step."""
    m, count, last = None, 0, 0
    for i, groups in enumerate(steps):
        top = max(scores[g].max() for g in groups)
        if m is None:
            m = top
        elif max(np.exp2(scores[g] - m).sum() for g in groups) > 2.0 ** 8 * 1.05:
            m, count, last = max(m, top), count + 1, i
    return count, last


@pytest.mark.parametrize("dim,layout", [(64, "NHD"), (128, "HND"), (256, "NHD")])
@pytest.mark.parametrize("new", [20, 40])
@pytest.mark.parametrize("splits", [1, -2])
def test_many_rows_whose_maximum_grows(kvq, dim, layout, new, splits):
    """80 and 160 rows per key head (one row tile and two, or two blocks at
    head size 256), up to eight tiles of 64 keys of which nearly every one
    exceeds the reference: O is rescaled again and again, and what it held
    before still counts for a twentieth, so that one rescaling missed among a
    request's last two is off by five tolerances or more."""
    b = growing_batch([(470, new), (0, new), (95, new), (170, new), (240, new)], dim, layout, 111, 0.56, 4)
    s = base_two_scores(b, 0, 0)
    count, last = growths(s, [[np.arange(i, min(i + 64, len(s)))] for i in range(0, len(s), 64)])
    assert count >= 5 and last >= 6
    assert growths(base_two_scores(b, 0, 3), [[np.arange(i, i + 64)] for i in range(0, 448, 64)])[0] == 0
    d = b.device()
    check(kvq.kvq_window_attention_nvfp4_per_head(**(dict(d, num_splits=splits) if splits > 0 else
                                                     through_workspace(kvq, d, -splits))), b.want())


@pytest.mark.parametrize("dim,layout", [(64, "HND"), (128, "NHD"), (256, "HND")])
@pytest.mark.parametrize("new", [1, 2])
@pytest.mark.parametrize("splits", [1, 3, -2])
def test_few_rows_whose_maximum_grows(kvq, dim, layout, new, splits):
    """4 and 8 rows per key head: a warp takes every fourth step of 32 keys
    and sums four keys of it per lane."""
    b = growing_batch([(660, new), (0, new), (200, new), (330, new)], dim, layout, 112, 0.5417, 3)
    s = base_two_scores(b, 0, 0)
    own = [[np.arange(i + r, i + 32, 8) for r in range(8)] for i in range(0, 640, 128)]         # the first warp's steps
    count, last = growths(s, own)
    assert count >= 3 and last >= 3
    d = b.device()
    check(kvq.kvq_window_attention_nvfp4_per_head(**(dict(d, num_splits=splits) if splits > 0 else
                                                     through_workspace(kvq, d, -splits))), b.want())


@pytest.mark.parametrize("dim", [64, 128])
def test_blocks_of_16_rows_whose_maximum_grows(kvq, dim):
    """480 requests on the same pages with the same four tokens: blocks of 16
    rows fill the GPU.  Every request has the first one's bits."""
    b = growing_batch([(660, 4)], dim, "NHD", 113, 0.5417, 3)
    d, n = b.device(), 480
    d.update(q=d["q"].repeat(n, 1, 1), query_start=torch.arange(0, 4 * n + 1, 4, dtype=torch.int32, device=DEV),
             seq_lens=d["seq_lens"].repeat(n), block_table=d["block_table"].repeat(n, 1), num_splits=1)
    out, lse = kvq.kvq_window_attention_nvfp4_per_head(**d)
    check((out[:4], lse[:4]), b.want())
    assert torch.equal(out.view(torch.int16), out[:4].view(torch.int16).repeat(n, 1, 1))
    assert torch.equal(lse, lse[:4].repeat(n, 1))


@pytest.mark.parametrize("dim,layout", [(64, "HND"), (128, "NHD"), (256, "NHD")])
@pytest.mark.parametrize("new", [30, 40])
def test_many_rows_over_more_tiles_than_mask_slots(kvq, dim, layout, new):
    """One range of 24 tiles of 64 keys (their existence masks go round a
    ring of 16 slots), with pages out of range behind position 1024 and a
    table that ends inside the sequence."""
    b = Batch([(1490, new), (1400, new)], 4, 1, dim, 16, layout, 114)
    b.table[0, [3, 66, 67, 81]] = [-1, 10 ** 6, -5, b.cache.raw.shape[1]]
    b.table[1, 70] = -1
    b.table = np.ascontiguousarray(b.table[:, :89])         # 1424 positions
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = kvq.kvq_window_attention_nvfp4_per_head(**b.device(), num_splits=1, status=status)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX
    check(got, b.want())


@pytest.mark.parametrize("dim,heads,kv", [(64, 4, 2), (128, 8, 2), (256, 4, 1)])
@pytest.mark.parametrize("new", [3, 40, 70])
@pytest.mark.parametrize("splits", [1, -2])
def test_tree_chain_has_the_windows_bits(kvq, dim, heads, kv, new, splits):
    """A tree that is one chain sees the keys that plain causal attention
    sees: both forms of mask give the same bits, in both kernels."""
    b = Batch([(77, new), (10, new), (0, new), (300, new)], heads, kv, dim, 16, "NHD", 115)
    rows = [[((2 << i) - 1) >> (64 * w) & (2 ** 64 - 1) for w in range(2)] for _, n in b.reqs for i in range(n)]
    d = through_workspace(kvq, b.device(), -splits) if splits < 0 else dict(b.device(), num_splits=splits)
    want = kvq.kvq_window_attention_nvfp4_per_head(**d)
    got = kvq.kvq_tree_attention_nvfp4_per_head(**d, tree_mask=mask_dev(rows))
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])
