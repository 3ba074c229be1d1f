"""Attention over whole prompts on the GPU against a plain 64-bit form
(tolerances derived there from the arithmetic), and a prompt with its
continuation: rotated and appended, attended as a prompt, then token by token
from the e4m3 cache."""
import numpy as np
import pytest
import torch

import fp8_per_head_reference as ref
from test_gpu_fp8_per_head import CANARY, DEV, bf16_dev, bits_of, check, dev, i32, kvq, pages_for   # noqa: F401

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
