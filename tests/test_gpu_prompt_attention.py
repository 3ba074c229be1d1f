"""Attention over whole prompts on the GPU against a plain 64-bit form
(tolerances derived there from the arithmetic), and a prompt with its
continuation: rotated and appended, attended as a prompt, then token by token
from the e4m3 cache."""
import numpy as np
import pytest
import torch

import fp8_per_head_reference as ref
from test_gpu_fp8_per_head import CANARY, DEV, Batch, attend, bf16_dev, bits_of, check, dev, i32, kvq, pages_for   # noqa: F401

pytestmark = pytest.mark.gpu


class Prompts:
    """Packed sequences, q, k and v slices of one packed projection, rows of no sequence behind the last one."""

    def __init__(self, lens, heads, kv_heads, dim, seed, pad=5, k_size=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.start = np.cumsum([0] + lens).tolist()
        T = self.start[-1] + pad
        self.split = (heads, heads + kv_heads)
        self.qkv = ref.to_bf16(rng.standard_normal((T, heads + 2 * kv_heads, dim)))
        self.qkv[:, self.split[0]:self.split[1]] = ref.to_bf16(
            ref.bf16(self.qkv[:, self.split[0]:self.split[1]]) * k_size)
        self.qkv[self.start[-1]:] = 0x7FC0                            # NaN behind the last sequence
        self.scale, self.max_len = dim ** -0.5, max(lens + [0])

    def parts(self, x):
        return x[:, :self.split[0]], x[:, self.split[0]:self.split[1]], x[:, self.split[1]:]

    def run(self, kvq, **over):
        q, k, v = self.parts(bf16_dev(self.qkv))
        call = dict(q=q, k=k, v=v, seq_start=i32(self.start), softmax_scale=self.scale, max_seq_len=self.max_len)
        return kvq.kvq_prompt_attention(**{**call, **over})

    def want(self, **mask):
        q, k, v = self.parts(ref.bf16(self.qkv))
        return ref.prompt_attention(q, k, v, self.start, self.scale, **mask)


def check_prompts(kvq, p, **mask):
    T, H = p.qkv.shape[0], p.split[0]
    out = bf16_dev(np.full((T, H, p.qkv.shape[2]), CANARY, np.uint16))
    lse = torch.full((T, H), 7.5, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = p.run(kvq, out=out, lse=lse, status=status, **{{"sinks": "num_sinks"}.get(k, k): v for k, v in mask.items()})
    assert int(status.item()) == 0
    live = p.start[-1]
    check(got, p.want(**mask), live)
    assert np.all(bits_of(out)[live:] == CANARY) and bool((lse[live:] == 7.5).all())


HEADS = [(64, 4, 2), (64, 7, 1), (128, 8, 2), (128, 3, 3), (128, 5, 1), (256, 4, 2), (256, 3, 1), (128, 16, 1)]


@pytest.mark.parametrize("dim,heads,kv", HEADS)
@pytest.mark.parametrize("lens", [[1], [5], [1, 2, 3, 0, 30], [128], [129, 64, 257], [300, 1, 0, 77]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (37, 4), (200, 300), (64, 140)])
def test_prompts(kvq, dim, heads, kv, lens, window, sinks):
    check_prompts(kvq, Prompts(lens, heads, kv, dim, 11 + dim + heads + len(lens)), window=window, sinks=sinks)


@pytest.mark.parametrize("dim,heads,kv", [(64, 8, 2), (128, 8, 2), (256, 2, 1)])
def test_a_long_prompt(kvq, dim, heads, kv):
    check_prompts(kvq, Prompts([1500, 700], heads, kv, dim, 23))


@pytest.mark.parametrize("dim,heads,kv", [(64, 40, 1), (128, 130, 1), (128, 300, 2), (256, 129, 1)])
def test_large_groups(kvq, dim, heads, kv):
    """More query heads per key head than a block has rows among them."""
    check_prompts(kvq, Prompts([33, 7], heads, kv, dim, 29))


def test_many_sequences(kvq):
    """More sequences than one look-up step takes, empty ones among them, at the ends too."""
    rng = np.random.default_rng(31)
    lens = [0, 0] + rng.integers(0, 12, 1500).tolist() + [0]
    check_prompts(kvq, Prompts(lens, 4, 2, 64, 31))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [6.0, 40.0])
def test_scores_that_grow(kvq, dim, size):
    """Keys that get larger along the sequence, so that references are left far behind."""
    p = Prompts([700, 130], 4, 2, dim, 37)
    ramp = np.linspace(0.05, size, p.qkv.shape[0])[:, None, None]
    k = slice(*p.split)
    p.qkv[:, k] = ref.to_bf16(ref.bf16(p.qkv[:, k]) * ramp)
    p.qkv[p.start[-1]:] = 0x7FC0
    check_prompts(kvq, p)
    check_prompts(kvq, p, window=150, sinks=3)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80])
def test_later_tokens_do_not_reach_earlier_rows(kvq, dim, bad):
    """NaN and infinities in a later token's key and value, in another sequence, and before the window."""
    p = Prompts([200, 150, 90], 4, 2, dim, 41)
    clean = p.run(kvq, window=100, num_sinks=2)
    want = p.want(window=100, sinks=2)
    at = [30, 170, 200, 300]                                          # tokens of the batch
    p.qkv[at, p.split[0]:] = bad
    got = p.run(kvq, window=100, num_sinks=2)
    out = ref.bf16(bits_of(got[0]))
    reach = np.zeros(p.start[-1], bool)
    for a in at:
        s = max(x for x in p.start if x <= a)
        e = min(x for x in p.start if x > a)
        reach[a:min(e, a + 100)] = True
        if a - s < 2:
            reach[a:e] = True
    ok = ~reach
    assert np.all(np.abs(out[:p.start[-1]][ok] - want[0][:p.start[-1]][ok]) <= want[2][:p.start[-1]][ok])
    rows = torch.from_numpy(np.flatnonzero(ok)).to(DEV)
    assert torch.equal(got[0][rows].view(torch.int16), clean[0][rows].view(torch.int16))
    assert not torch.isfinite(got[1][at]).all()


def test_strides_scales_and_no_lse(kvq):
    p = Prompts([130, 40], 6, 2, 64, 43, pad=0)
    T = p.qkv.shape[0]
    q, k, v = p.parts(bf16_dev(p.qkv))
    outs = torch.zeros((T, 9, 64), dtype=torch.bfloat16, device=DEV)
    lses = torch.zeros((T, 11), device=DEV)
    got = p.run(kvq, q=q.contiguous(), k=k.transpose(0, 1).contiguous().transpose(0, 1), out=outs[:, 1:7], lse=lses[:, 3:9])
    check(got, p.want())
    assert bool((outs[:, 0] == 0).all()) and bool((outs[:, 7:] == 0).all()) and bool((lses[:, :3] == 0).all())
    out, lse = p.run(kvq, lse=False)
    assert lse is None and torch.equal(out, got[0])
    for scale in (0.0, -0.3):
        p.scale = scale
        check(p.run(kvq), p.want())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [2.0 ** 78, 2.0 ** -60])
def test_values_far_from_one(kvq, dim, size):
    """Sums over large values stay finite behind a reference that is far off; small ones keep their precision."""
    p = Prompts([600, 130], 4, 2, dim, 45)
    ramp = np.linspace(0.05, 12.0, p.qkv.shape[0])[:, None, None]
    k, v = slice(*p.split), slice(p.split[1], None)
    p.qkv[:, k] = ref.to_bf16(ref.bf16(p.qkv[:, k]) * ramp)
    p.qkv[:, v] = ref.to_bf16(np.clip(ref.bf16(p.qkv[:, v]), -1, 1) * size)
    p.qkv[p.start[-1]:] = 0x7FC0
    check_prompts(kvq, p)


def test_bad_sequences_are_skipped(kvq):
    p = Prompts([60, 50, 70, 40], 4, 2, 128, 47)
    want = p.want()
    T = p.qkv.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = bf16_dev(np.full((T, 4, 128), CANARY, np.uint16))
    got = p.run(kvq, out=out, status=status, max_seq_len=60)          # the third is too long
    assert int(status.item()) == kvq.STATUS_BAD_BATCH
    keep = np.r_[0:110, 180:220]
    o = ref.bf16(bits_of(got[0]))
    assert np.all(np.abs(o[keep] - want[0][keep]) <= want[2][keep])
    assert np.all(bits_of(out)[110:180] == CANARY) and np.all(bits_of(out)[220:] == CANARY)
    for start in ([0, 60, T + 1], [-5, 60], [0, 60, 30, 40]):
        status.zero_()
        p.run(kvq, seq_start=i32(start), status=status, max_seq_len=T)
        torch.cuda.synchronize()
        assert int(status.item()) == kvq.STATUS_BAD_BATCH


def test_nothing_to_do(kvq):
    p = Prompts([0, 0], 4, 2, 64, 53)
    check_prompts(kvq, p)
    out, lse = p.run(kvq, seq_start=i32([0]))
    assert out.shape == (5, 4, 64)
    empty = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    out, lse = kvq.kvq_prompt_attention(empty, empty[:, :2], empty[:, :2], i32([0, 0]), 0.1, 0)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("lens", [[20, 9], [400, 90]])
def test_graphs_streams_and_repeats(kvq, lens):
    p = Prompts(lens, 8, 2, 128, 59, pad=0)
    want = p.run(kvq)
    for _ in range(3):
        got = p.run(kvq)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = p.run(kvq, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qkv = bf16_dev(p.qkv)
    q, k, v = p.parts(qkv)
    start = i32(p.start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = kvq.kvq_prompt_attention(q, k, v, start, p.scale, p.max_len)
        twice = kvq.kvq_prompt_attention(inside[0], k, v, start, p.scale, p.max_len)
    qkv.copy_(qkv.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    again = kvq.kvq_prompt_attention(q, k, v, start, p.scale, p.max_len)
    assert torch.equal(inside[0], again[0]) and torch.equal(inside[1], again[1])
    more = kvq.kvq_prompt_attention(again[0], k, v, start, p.scale, p.max_len)
    assert torch.equal(twice[0], more[0])


def test_refuses_what_does_not_fit(kvq):
    p = Prompts([30], 4, 2, 64, 61)
    q, k, v = p.parts(bf16_dev(p.qkv))

    def refused(kind, match, **over):
        with pytest.raises(kind, match=match):
            p.run(kvq, **over)

    refused(ValueError, "q", q=q.float())
    refused(ValueError, "k", k=k[:-1])
    refused(ValueError, "v", v=v[..., :32])
    refused(ValueError, "k", k=k.cpu())
    refused(ValueError, "seq_start", seq_start=i32(p.start).long())
    refused(ValueError, "seq_start", seq_start=i32([]))
    refused(ValueError, "out", out=torch.empty((3, 4, 64), dtype=torch.bfloat16, device=DEV))
    refused(ValueError, "lse", lse=torch.empty((35, 4), dtype=torch.bfloat16, device=DEV))
    refused(RuntimeError, "num_heads", q=q[:, :3])
    refused(RuntimeError, "softmax_scale", softmax_scale=float("inf"))
    refused(RuntimeError, "num_sinks", num_sinks=-1)
    refused(RuntimeError, "max_seq_len", max_seq_len=-1)
    refused(RuntimeError, "strides", k=k[:1].expand(35, 2, 64))


# --------------------------------------------------------------------------
# the operators together
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dim,heads,kv,layout,block,rot,interleaved,window,sinks", [
    (64, 7, 1, "HND", 24, 32, True, 0, 0), (128, 8, 2, "NHD", 16, 128, False, 50, 3), (256, 4, 2, "NHD", 32, 64, False, 0, 0)])
def test_prompts_chunks_and_decoded_tokens(kvq, dim, heads, kv, layout, block, rot, interleaved, window, sinks):
    """Prompts are rotated, appended and attended whole; then a chunk of tokens and single ones over the cache."""
    rng = np.random.default_rng(67 + dim)
    steps = [[90, 37, 150], [40, 3, 21]] + [[1, 1, 1]] * 5
    total, table = pages_for([(0, sum(s[b] for s in steps)) for b in range(3)], block, rng)
    cache = ref.Cache(total, block, kv, dim, layout, rng)
    raw, scales, block_table = dev(cache.raw()), dev(cache.scales), dev(table.astype(np.int32))
    angle = rng.uniform(-7, 7, (300, rot // 2))
    cos_sin = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    scale, lens = dim ** -0.5, [0, 0, 0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for step, new in enumerate(steps):
        start = np.cumsum([0] + new).tolist()
        positions = np.concatenate([np.arange(c, c + n) for c, n in zip(lens, new)])
        lens = [c + n for c, n in zip(lens, new)]
        x = ref.to_bf16(rng.standard_normal((start[-1], heads + 2 * kv, dim)))
        q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
        on = bf16_dev(x)
        begin, seq_lens, most = i32(start), i32(lens), max(new)
        rq, rk = kvq.kvq_rope_append_fp8_per_head(
            on[:, :heads], on[:, heads:heads + kv], on[:, heads + kv:], dev(positions), dev(cos_sin), begin, seq_lens,
            block_table, raw, scales, most, interleaved=interleaved, layout=layout, status=status)
        if step == 0:
            got = kvq.kvq_prompt_attention(rq, rk, on[:, heads + kv:], begin, scale, most, window=window, num_sinks=sinks,
                                           status=status)
        else:
            got = kvq.kvq_window_attention_fp8_per_head(rq, begin, seq_lens, block_table, raw, scales, scale, most, max(lens),
                                                        window=window, num_sinks=sinks, layout=layout, status=status)
        want_q, want_k = np.zeros_like(q), np.zeros_like(k)
        assert ref.append(cache, q, k, v, positions, cos_sin, start, lens, table, interleaved, want_q, want_k) == 0
        assert np.array_equal(bits_of(rq), want_q) and np.array_equal(bits_of(rk), want_k)
        assert np.array_equal(cache.from_raw(raw.cpu().numpy()), cache.codes)
        assert np.array_equal(scales.cpu().numpy(), cache.scales)
        if step == 0:
            want = ref.prompt_attention(ref.bf16(want_q), ref.bf16(want_k), ref.bf16(v), start, scale, window, sinks)
        else:
            want = ref.cached_attention(cache, ref.bf16(want_q), start, lens, table, scale, window, sinks)
        check(got, want)
        assert int(status.item()) == 0


def test_values_the_cache_holds_exactly(kvq):
    """Keys and values of e4m3's own: a prompt whole and in parts over the cache agree with one 64-bit form."""
    rng = np.random.default_rng(71)
    n, first, heads, kv, dim, block = 230, 100, 8, 2, 128, 16
    total, table = pages_for([(0, n)], block, rng)
    raw = torch.zeros((total, 2, block, kv, dim), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((total, 2, kv), dtype=torch.uint8, device=DEV)
    values = np.array([0.0, 0.25, -0.5, 1.0, -1.75, 3.5, -3.5])                    # 3.5 = 448 * 2^-7
    q = ref.to_bf16(rng.standard_normal((n, heads, dim)))
    k, v = (ref.to_bf16(rng.choice(values, (n, kv, dim))) for _ in range(2))
    k[:, :, 0] = v[:, :, 0] = ref.to_bf16(np.float32(3.5))                        # every page's scale: the same
    on = [bf16_dev(x) for x in (q, k, v)]
    still = torch.tensor([[1.0] * 8 + [0.0] * 8], device=DEV).repeat(n, 1).contiguous()
    block_table, where = dev(table.astype(np.int32)), torch.arange(n, device=DEV)
    want = ref.prompt_attention(*(ref.bf16(x) for x in (q, k, v)), [0, n], dim ** -0.5)
    check(kvq.kvq_prompt_attention(*on, i32([0, n]), dim ** -0.5, n), want)
    got = []
    for t0, t1 in [(0, first), (first, n - 3)] + [(t, t + 1) for t in range(n - 3, n)]:
        rq, rk = kvq.kvq_rope_append_fp8_per_head(*(x[t0:t1] for x in on), where[t0:t1], still, i32([0, t1 - t0]), i32([t1]),
                                                  block_table, raw, scales, t1 - t0)
        assert torch.equal(rq, on[0][t0:t1]) and torch.equal(rk, on[1][t0:t1])
        got.append(kvq.kvq_window_attention_fp8_per_head(rq, i32([0, t1 - t0]), i32([t1]), block_table, raw, scales,
                                                         dim ** -0.5, t1 - t0, t1))
    # (weights rounded more finely than the prompt's: the same tolerances hold)
    check([torch.cat([g[i] for g in got]) for i in range(2)], want)


def test_large_calls_gather_by_default(kvq):
    b = Batch([(200, 130), (17, 130), (0, 130), (90, 101)], 64, 8, 64, 16, "NHD", 73)
    call = b.device()
    assert kvq.kvq_fp8_attention_default_splits(130, 64, 8, 64, 4, max(b.lens)) == (1, True)
    want = b.want(gathered=True)
    got = attend(kvq, call, None)
    check(got, want)
    # a bound on the lengths that is far off costs nothing: the block table's reach holds as well
    loose = attend(kvq, dict(call, max_seq_len=(1 << 31) - 1), None)
    assert torch.equal(loose[0], got[0]) and torch.equal(loose[1], got[1])
    loose = attend(kvq, dict(call, max_query_len=100000), None)
    assert torch.equal(loose[0], got[0]) and torch.equal(loose[1], got[1])
    # queries that the copy engine cannot address: decoded in the attention
    same = call["q"][:1].expand(b.q_bits.shape[0], -1, -1)
    b.q_bits[:] = b.q_bits[:1]
    check(attend(kvq, dict(call, q=same), None), b.want())


def test_calls_at_once(kvq):
    """Every operator on two streams at the same time, each call with its own outputs and workspace."""
    b = Batch([(2000, 130), (700, 130), (40, 130), (900, 101)], 64, 8, 64, 16, "NHD", 79)
    few = Batch([(3000, 1), (500, 1)], 64, 8, 64, 16, "NHD", 83)
    p = Prompts([500, 300], 64, 8, 64, 89, pad=0)
    big, small = b.device(), few.device()
    jobs = [lambda s: attend(kvq, dict(big, stream=s), None), lambda s: attend(kvq, dict(small, stream=s), None),
            lambda s: attend(kvq, dict(big, stream=s), 2), lambda s: p.run(kvq, stream=s)]
    want = [f(None) for f in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(4):
        for i, f in enumerate(jobs):
            got.append((i, f(streams[(i + turn) % 2])))
            got.append((i, f(streams[(i + turn + 1) % 2])))
    torch.cuda.synchronize()
    for i, g in got:
        assert torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1])


def test_graphs_that_share_a_workspace(kvq):
    one, two = (Batch(reqs, 8, 2, 128, 16, "NHD", 97 + len(reqs)) for reqs in ([(300, 90), (20, 64)], [(5, 90), (600, 90), (0, 90)]))
    calls, need = [b.device() for b in (one, two)], 0
    for c in calls:
        need = max(need, kvq.kvq_fp8_attention_workspace_bytes(c["q"].shape[0], 8, 2, 128, 2, c["max_query_len"], c["max_seq_len"]))
    held = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    want = [kvq.kvq_window_attention_fp8_per_head(**c, num_splits=1, workspace=held) for c in calls]
    graphs, inside = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            inside.append(kvq.kvq_window_attention_fp8_per_head(**c, num_splits=1, workspace=held))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for got, w in zip(inside, want):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
        for got in inside:
            got[0].zero_()
