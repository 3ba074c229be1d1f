"""Serving from the per-head e4m3 cache on the GPU: the append of rotated keys
and values against the definition's fp32 steps, byte for byte, untouched bytes
among them, and the attention over the cache against a plain 64-bit form
(tolerances derived there from the arithmetic)."""
import numpy as np
import pytest
import torch

import fp8_per_head_reference as ref

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


def pages_for(reqs, block, rng, spare=3):
    """A shuffled block table for requests (context, new), one column wider than needed."""
    need = [max(1, -(-(c + n) // block)) for c, n in reqs]
    total = sum(need) + spare
    order = rng.permutation(total)
    table = np.full((len(reqs), max(need, default=0) + 1), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return total, table


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------

class Append:
    """New tokens of requests (context, new), with padding rows behind the last one."""

    def __init__(self, reqs, heads, kv_heads, dim, block, layout, rot, seed, interleaved=False, size=1.0, pad=3,
                 max_pos=1000):
        rng = self.rng = np.random.default_rng(seed)
        self.reqs, self.interleaved, self.layout, self.heads = reqs, interleaved, layout, heads
        self.lens = [c + n for c, n in reqs]
        self.start = np.cumsum([0] + [n for _, n in reqs]).tolist()
        total, self.table = pages_for(reqs, block, rng)
        self.cache = ref.Cache(total, block, kv_heads, dim, layout, rng)
        T = self.T = self.start[-1] + pad
        # one packed projection, so that heads and tokens are strided
        self.qkv = ref.to_bf16(rng.standard_normal((T, heads + 2 * kv_heads, dim)) * size)
        self.positions = rng.integers(0, max_pos, T)
        angle = rng.uniform(-7, 7, (max_pos, rot // 2))
        self.cos_sin = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32).reshape(max_pos, rot)
        self.split = (heads, heads + kv_heads)

    def parts(self, x):
        return x[:, :self.split[0]], x[:, self.split[0]:self.split[1]], x[:, self.split[1]:]

    def run(self, kvq, status=None, in_place=False, no_q=False, no_k=False, stream=None, cos_sin=None, most=None):
        """(q_out bits, k_out bits, codes, scales) of the call; outputs that it leaves alone hold CANARY."""
        qkv = bf16_dev(self.qkv)
        q, k, v = self.parts(qkv)
        cache, scales = dev(self.cache.raw()), dev(self.cache.scales)
        if in_place:
            qo, ko = q, k
        else:
            qo = bf16_dev(np.full(q.shape, CANARY, np.uint16))
            ko = bf16_dev(np.full(k.shape, CANARY, np.uint16))
        got = kvq.kvq_rope_append_fp8_per_head(
            None if no_q else q, k, v, dev(self.positions), dev(self.cos_sin) if cos_sin is None else cos_sin,
            i32(self.start), i32(self.lens), dev(self.table.astype(np.int32)), cache, scales, max([n for _, n in self.reqs] + [0]) if most is None else most,
            interleaved=self.interleaved, layout=self.layout, q_out=qo, k_out=False if no_k else ko, status=status,
            stream=stream)
        torch.cuda.synchronize()
        assert (got[0] is None) == no_q and (got[1] is None) == no_k
        return bits_of(qo), bits_of(ko), self.cache.from_raw(cache.cpu().numpy()), scales.cpu().numpy()

    def want(self, in_place=False):
        q, k, v = self.parts(self.qkv)
        qo = q.copy() if in_place else np.full(q.shape, CANARY, np.uint16)
        ko = k.copy() if in_place else np.full(k.shape, CANARY, np.uint16)
        status = ref.append(self.cache, q, k, v, self.positions, self.cos_sin, self.start, self.lens, self.table,
                            self.interleaved, qo, ko)
        return qo, ko, self.cache.codes, self.cache.scales, status


def check_append(kvq, case, **how):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = case.run(kvq, status=status, **how)
    qo, ko, codes, scales, bits = case.want(how.get("in_place", False))
    assert int(status.item()) == bits
    assert np.array_equal(got[3], scales), "scales differ"
    bad = got[2] != codes
    assert not bad.any(), f"{int(bad.sum())} codes differ, first at {np.argwhere(bad)[0]}"
    if not how.get("no_q"):
        assert np.array_equal(got[0], qo)
    if not how.get("no_k"):
        assert np.array_equal(got[1], ko)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (64, 32, True), (128, 128, False), (128, 64, True),
                                                 (256, 256, True), (256, 32, False), (128, 0, False)])
@pytest.mark.parametrize("block", [1, 16, 24, 64])
def test_append_bytes(kvq, dim, rot, interleaved, block, layout):
    reqs = [(0, 1), (37, 1), (block, 2), (5, 70), (block - 1, 1), (130, 17), (3, 0), (0, block), (2 * block, block + 1)]
    check_append(kvq, Append(reqs, 6, 2, dim, block, layout, rot, 100 + dim + rot + block, interleaved))


@pytest.mark.parametrize("size", [1e-30, 1e-12, 3e-3, 300.0, 1e15, 3e38])
def test_append_of_any_magnitude(kvq, size):
    """Scales of any size, growing past and staying below what the pages hold, clamped at both ends."""
    case = Append([(37, 5), (16, 1), (40, 200), (7, 3)], 4, 2, 64, 16, "NHD", 64, 7, size=min(size, 1e30))
    if size > 1e30:
        case.qkv[::5] = 0x7F7F                                       # the largest bf16
        case.cos_sin[:] = np.concatenate([np.ones((1000, 32)), np.zeros((1000, 32))], 1)   # no sum overflows
    check_append(kvq, case)


def test_append_recodes_what_the_page_holds(kvq):
    """Codes of every kind under a scale that grows by 1 to 8 powers of two, subnormals and NaN among them."""
    case = Append([(100, 28)] * 8, 2, 2, 128, 128, "NHD", 128, 11, size=1.0)
    for b in range(8):
        page = case.table[b, 0]
        case.cache.codes[page, :, :100].reshape(-1)[:] = np.resize(np.arange(256, dtype=np.uint8), 2 * 100 * 2 * 128)
        case.cache.scales[page] = 127 - 7 - b
    check_append(kvq, case)


def test_append_zeros_signs_and_exact_ties(kvq):
    """Zeros of both signs keep them (rotated and not), pages of zeros get the least scale, and values half way
    between two codes go to the even one."""
    case = Append([(0, 40), (8, 8)], 2, 1, 64, 16, "HND", 0, 12)
    case.qkv[:16] = np.resize(np.array([0, 0x8000], np.uint16), case.qkv[:16].shape)
    grid = ref.MAGNITUDE
    mid = (grid[:-1] + grid[1:]) / 2                                  # exact in bf16: 5 significant bits
    case.qkv[16:32] = ref.to_bf16(np.resize(np.concatenate([mid, -mid, [448.0]]), case.qkv[16:32].shape))
    check_append(kvq, case)


@pytest.mark.parametrize("how", [dict(in_place=True), dict(no_q=True), dict(no_k=True), dict(no_q=True, no_k=True)])
def test_append_outputs_in_place_or_left_out(kvq, how):
    check_append(kvq, Append([(9, 3), (0, 50)], 4, 2, 128, 16, "NHD", 64, 13), **how)


def test_append_skips_bad_tokens_pages_and_requests(kvq):
    case = Append([(5, 3), (10, 30), (0, 4), (2, 6), (1, 1)], 4, 2, 64, 16, "NHD", 64, 14)
    case.positions[1] = -1                                            # one token's position below the table
    case.positions[20] = 1000                                         # and one past it
    case.table[1, 1] = case.cache.codes.shape[0]                      # a page that does not exist
    case.table[2, 0] = -7
    case.lens[3] = 5                                                  # more new tokens than positions
    case.lens[4] = -3
    check_append(kvq, case)


def test_append_past_the_block_table(kvq):
    case = Append([(5, 60)], 4, 2, 64, 16, "NHD", 64, 15)
    case.table = case.table[:, :2].copy()
    check_append(kvq, case)


@pytest.mark.parametrize("block,new", [(16, 3), (16, 40), (64, 200), (24, 1), (1024, 600)])
def test_append_at_the_last_positions_of_all(kvq, block, new):
    """Sequences that end at and next to the largest length, far past their block tables: nothing is appended, and
    rotated rows are written as ever."""
    case = Append([(5, new), (0, new), (9, new)], 4, 2, 64, block, "NHD", 64, 21)
    case.lens[:2] = [(1 << 31) - 1, (1 << 31) - 1 - new // 2]
    check_append(kvq, case)


def test_append_with_a_loose_bound(kvq):
    """max_query_len far above what any request brings."""
    check_append(kvq, Append([(5, 3), (70, 21), (0, 0)], 4, 2, 128, 16, "NHD", 128, 20), most=100000)


def test_append_of_nothing(kvq):
    for reqs in ([], [(3, 0), (0, 0)]):
        case = Append(reqs, 2, 1, 64, 16, "NHD", 64, 16)
        got = case.run(kvq)
        assert np.all(got[0] == CANARY) and np.all(got[1] == CANARY)
        assert np.array_equal(got[2], case.cache.codes) and np.array_equal(got[3], case.cache.scales)


def test_append_many_heads_and_a_full_grid(kvq):
    """Enough tokens that a lane group takes eight query heads, with heads left over."""
    check_append(kvq, Append([(3, 700), (60, 500)], 13, 1, 128, 64, "NHD", 128, 17))


def test_append_twice_and_token_by_token(kvq):
    """A repeated call changes nothing more; appending token by token leaves the scales of appending at once."""
    reqs = [(30, 20), (0, 33)]
    case = Append(reqs, 2, 2, 64, 16, "NHD", 64, 18, pad=0)
    once = case.run(kvq)
    case.cache.codes, case.cache.scales = once[2].copy(), once[3].copy()
    again = case.run(kvq)
    assert all(np.array_equal(x, y) for x, y in zip(once, again))
    case = Append(reqs, 2, 2, 64, 16, "NHD", 64, 18, pad=0)
    cache, scales = dev(case.cache.raw()), dev(case.cache.scales)
    q, k, v = case.parts(bf16_dev(case.qkv))
    for i in range(33):
        rows = [case.start[b] + i for b, (_, n) in enumerate(reqs) if i < n]
        live = [b for b, (_, n) in enumerate(reqs) if i < n]
        pick = torch.tensor(rows, device=DEV)
        kvq.kvq_rope_append_fp8_per_head(
            q[pick], k[pick], v[pick], dev(case.positions)[pick], dev(case.cos_sin), i32(list(range(len(rows) + 1))),
            i32([reqs[b][0] + i + 1 for b in live]), dev(case.table[live].astype(np.int32)), cache, scales, 1)
    assert np.array_equal(scales.cpu().numpy(), once[3])
    # codes differ at most where an entry was rounded twice, in e4m3's subnormals
    diff = case.cache.from_raw(cache.cpu().numpy()) != once[2]
    assert np.all((once[2][diff] & 0x7F) <= 8)


def test_append_on_another_stream_and_in_a_graph(kvq):
    case = Append([(5, 3), (70, 1)], 4, 2, 128, 16, "NHD", 128, 19, pad=0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = case.run(kvq, stream=side)
    q, k, v = case.parts(bf16_dev(case.qkv))
    cache, scales = dev(case.cache.raw()), dev(case.cache.scales)
    args = (q, k, v, dev(case.positions), dev(case.cos_sin), i32(case.start), i32(case.lens), dev(case.table.astype(np.int32)),
            cache, scales, 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo, ko = kvq.kvq_rope_append_fp8_per_head(*args)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits_of(qo), got[0]) and np.array_equal(bits_of(ko), got[1])
    assert np.array_equal(case.cache.from_raw(cache.cpu().numpy()), got[2])
    assert np.array_equal(scales.cpu().numpy(), got[3])


# --------------------------------------------------------------------------
# attention over the cache
# --------------------------------------------------------------------------

def through_workspace(kvq, call, splits):
    """The arguments of a call whose ranges join through a workspace, not in clusters."""
    T, H, D = call["q"].shape
    need = max(16, kvq.kvq_per_head_attention_workspace_bytes(T, H, D, splits))
    return dict(call, num_splits=splits, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))


class Batch:
    """Requests with (context, new tokens), a shuffled block table, queries."""

    def __init__(self, reqs, heads, kv_heads, dim, block, layout, seed, extra_tokens=0, q_scale=1.0, exponents=(-9, -6)):
        rng = np.random.default_rng(seed)
        self.reqs, self.rng, self.layout = reqs, rng, layout
        self.lens = [c + n for c, n in reqs]
        self.start = np.cumsum([0] + [n for _, n in reqs]).tolist()
        total, self.table = pages_for(reqs, block, rng)
        self.cache = ref.Cache(total, block, kv_heads, dim, layout, rng, exponents)
        T = self.start[-1] + extra_tokens
        self.q_bits = ref.to_bf16(rng.standard_normal((T, heads, dim)) * q_scale)
        self.scale = dim ** -0.5

    def device(self):
        return dict(q=bf16_dev(self.q_bits), query_start=i32(self.start), seq_lens=i32(self.lens),
                    block_table=dev(self.table.astype(np.int32)), kv_cache=dev(self.cache.raw()),
                    kv_scales=dev(self.cache.scales), softmax_scale=self.scale,
                    max_query_len=max([n for _, n in self.reqs] + [0]), max_seq_len=max(self.lens + [0]),
                    layout=self.layout)

    def want(self, **mask):
        return ref.cached_attention(self.cache, ref.bf16(self.q_bits), self.start, self.lens, self.table, self.scale, **mask)


def gathering(kvq, call, requests, **mask):
    """The arguments of a call that gathers its entries, so many requests at a time."""
    (T, H, D), pages = call["q"].shape, call["kv_scales"]
    need = kvq.kvq_fp8_attention_workspace_bytes(T, H, pages.shape[2], D, requests, call["max_query_len"],
                                                 call["max_seq_len"], mask.get("window", 0), mask.get("num_sinks", 0))
    assert need > 0
    # NaN wherever nothing is written
    return dict(call, num_splits=1, workspace=torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV))


def attend(kvq, call, splits, **mask):
    """splits < 0: through a workspace; None: the default; "gather": two requests' entries at a time."""
    if splits == "gather":
        call = gathering(kvq, call, 2, **mask)
    elif splits is not None:
        call = dict(call, num_splits=splits) if splits > 0 else through_workspace(kvq, call, -splits)
    return kvq.kvq_window_attention_fp8_per_head(**call, **mask)


def check(got, want, rows=None):
    out, lse, tol_o, tol_l = want
    o, l = ref.bf16(bits_of(got[0])), got[1].cpu().numpy().astype(np.float64)
    sl = slice(0, rows)
    err = np.abs(o[sl] - out[sl])
    assert np.all(err <= tol_o[sl]), f"out: worst error / tolerance {np.nanmax(err / tol_o[sl])}"
    dead = np.isneginf(lse[sl])
    assert np.array_equal(np.isneginf(l[sl]), dead)
    le = np.abs(l[sl][~dead] - lse[sl][~dead])
    assert np.all(le <= tol_l[sl][~dead]), f"lse: worst error / tolerance {np.max(le / tol_l[sl][~dead])}"


SHAPES = [(64, "NHD", 4, 2, 16), (64, "HND", 7, 1, 24), (128, "NHD", 8, 2, 16), (128, "HND", 6, 3, 64), (128, "NHD", 5, 5, 1),
          (256, "NHD", 4, 2, 32), (256, "HND", 3, 1, 24), (128, "HND", 32, 1, 48)]


@pytest.mark.parametrize("dim,layout,heads,kv,block", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (37, 4), (64, 40), (500, 1000)])
@pytest.mark.parametrize("splits", [1, 3, -3, None])
def test_decode(kvq, dim, layout, heads, kv, block, window, sinks, splits):
    b = Batch([(0, 1), (31, 1), (32, 1), (300, 1), (129, 1), (1, 1)], heads, kv, dim, block, layout, 31 + dim + block)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = attend(kvq, b.device(), splits, window=window, num_sinks=sinks, status=status)
    check(got, b.want(window=window, sinks=sinks))
    assert int(status.item()) == 0


@pytest.mark.parametrize("dim,layout,heads,kv,block", SHAPES)
@pytest.mark.parametrize("window,sinks,splits", [(0, 0, 1), (0, 0, -2), (29, 5, 1), (29, 5, -3), (100, 0, None),
                                                 (0, 0, "gather"), (29, 5, "gather"), (1, 70, "gather"), (70, 100, "gather")])
def test_chunks(kvq, dim, layout, heads, kv, block, window, sinks, splits):
    b = Batch([(0, 70), (65, 33), (200, 1), (7, 64), (0, 0), (130, 129)], heads, kv, dim, block, layout, 57 + dim + block)
    check(attend(kvq, b.device(), splits, window=window, num_sinks=sinks),
          b.want(window=window, sinks=sinks, gathered=splits == "gather"))


def skip_unless(splits, rows):
    if splits == "gather" and rows <= 48:
        pytest.skip("few rows are not gathered for")
    if splits not in ("gather", None) and splits > 1 and rows > 32:
        pytest.skip("clusters take few rows")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("block", [8, 16, 64])
@pytest.mark.parametrize("new", [1, 3, 40, 70])
@pytest.mark.parametrize("splits", [1, 3, -2, "gather"])
def test_scales_far_apart(kvq, dim, block, new, splits):
    """Pages whose scales differ by up to 2^30 either way, so that the references rise and fall."""
    skip_unless(splits, 4 * new)
    b = Batch([(700, new), (63, new)], 4, 1, dim, block, "NHD", 71 + dim + block + new)
    pages = b.cache.scales.shape[0]
    b.cache.scales[:, 0] = (127 - 7 + b.rng.integers(-3, 2, (pages, 1))).astype(np.uint8)
    b.cache.scales[:, 1] = (127 - 7 + b.rng.choice([0, 0, 1, -1, 5, 9, -8, 15, -15], (pages, 1))).astype(np.uint8)
    check(attend(kvq, b.device(), splits), b.want(gathered=splits == "gather"))


@pytest.mark.parametrize("new,splits", [(1, None), (70, None), (70, "gather")])
def test_scales_at_and_past_the_ends(kvq, new, splits):
    """The least and the largest scale, and bytes outside them, which read as the nearer one."""
    b = Batch([(200, new), (90, new)], 4, 2, 128, 16, "HND", 83, q_scale=1.0)
    pages = b.cache.scales.shape[0]
    b.cache.scales[:, 0] = 127 - 9
    gathered = splits == "gather"
    b.cache.scales[:, 1] = b.rng.choice([0, 66, 67, 70], (pages, 2)).astype(np.uint8)
    check(attend(kvq, b.device(), splits), b.want(gathered=gathered))
    b.cache.scales[:, 1] = b.rng.choice([255, 188, 187, 180], (pages, 2)).astype(np.uint8)
    check(attend(kvq, b.device(), splits), b.want(gathered=gathered))
    b.cache.scales[:, 0] = b.rng.choice([0, 67, 80], (pages, 2)).astype(np.uint8)     # scores of about zero
    check(attend(kvq, b.device(), splits, window=50), b.want(window=50, gathered=gathered))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,splits", [(1, None), (1, 1), (3, -2), (70, 1), (70, None), (70, "gather")])
def test_the_largest_scale_before_the_least(kvq, dim, new, splits):
    """Pages of huge values before pages of zeros, whose scale is the least: sums stay finite, either way round."""
    b = Batch([(600, new), (700, new)], 4, 1, dim, 16, "NHD", 87)
    b.cache.scales[:, 0] = 127 - 9
    codes = b.cache.codes.copy()
    for order in (1, -1):
        b.cache.codes[:] = codes
        for r, n in enumerate(b.lens):
            used = b.table[r][:-(-n // 16)][::order]
            b.cache.scales[used, 1] = np.where(np.arange(len(used)) < len(used) // 2, 187, 67)[:, None]
            b.cache.codes[used[len(used) // 2:], 1] = 0
        want = b.want(gathered=splits == "gather")
        assert np.abs(want[0]).max() > 2.0 ** 60
        check(attend(kvq, b.device(), splits), want)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,splits", [(1, None), (1, 1), (70, 1), (70, "gather")])
def test_subnormal_codes(kvq, dim, new, splits):
    """Codes below e4m3's normal range alone, either zero among them."""
    b = Batch([(200, new), (33, new)], 4, 2, dim, 16, "NHD", 85, exponents=(-3, 8))
    b.cache.codes &= 0x87
    b.scale = 4.0
    check(attend(kvq, b.device(), splits), b.want(gathered=splits == "gather"))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,splits", [(4, None), (4, 1), (4, -3), (70, 1), (70, None), (70, -2), (70, "gather")])
@pytest.mark.parametrize("block", [1, 16])
def test_hidden_pages_of_any_scale_have_no_effect(kvq, dim, new, splits, block):
    """Keys and values as large as the cache holds, where earlier tokens do not see them yet and later ones no longer do."""
    b = Batch([(90, new), (33, new)], 4, 1, dim, block, "NHD", 89)
    mask = dict(window=60, num_sinks=2)
    clean = attend(kvq, b.device(), splits, **mask)
    want = b.want(window=60, sinks=2, gathered=splits == "gather")
    sees = np.ones(b.start[-1], bool)
    for r, n in enumerate(b.lens):
        first = n - new
        cols = [(first - 60 + new // 2) // block - (block > 1)]       # no longer seen by about half of the new tokens
        if block < new:
            cols.append((n - 2) // block)                             # not seen yet by most of them
        for col in cols:
            if col * block < 2:                                       # (sinks stay visible)
                continue
            b.cache.scales[b.table[r][col]] = 187
            for i in range(new):
                if first + i - 60 < (col + 1) * block - 1 and col * block <= first + i:
                    sees[b.start[r] + i] = False
    assert sees.any() and not sees.all()
    got = attend(kvq, b.device(), splits, **mask)
    check((clean[0], clean[1]), want)
    rows = np.flatnonzero(sees)
    err = np.abs(ref.bf16(bits_of(got[0]))[rows] - want[0][rows])
    assert np.all(err <= want[2][rows]), f"worst error / tolerance {np.max(err / want[2][rows])}"
    le = np.abs(got[1].cpu().numpy().astype(np.float64)[rows] - want[1][rows])
    assert np.all(le <= want[3][rows])


@pytest.mark.parametrize("new", [1, 130])
@pytest.mark.parametrize("splits", [1, 5, -5, "gather"])
def test_padded_requests_see_nothing_and_other_rows_are_left(kvq, new, splits):
    skip_unless(splits, 4 * new)
    b = Batch([(50, new), (0, new), (90, new)], 8, 2, 128, 16, "NHD", 91, extra_tokens=5)
    b.lens[1] = 0                                                     # its queries have negative positions
    b.lens[0] = new // 2                                              # and half of these (one token: none)
    call = b.device()
    out = bf16_dev(np.full(b.q_bits.shape, CANARY, np.uint16))
    lse = torch.full(b.q_bits.shape[:2], 7.5, device=DEV)
    got = attend(kvq, dict(call, out=out, lse=lse), splits)
    live = b.start[-1]
    check(got, b.want(gathered=splits == "gather"), live)
    assert np.all(bits_of(out)[live:] == CANARY) and bool((lse[live:] == 7.5).all())
    assert bool((out[b.start[1]:b.start[2]] == 0).all()) and bool(torch.isneginf(lse[b.start[1]:b.start[2]]).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("splits", [1, -4, "gather"])
def test_hidden_entries_have_no_effect(kvq, dim, new, splits):
    """NaN codes wherever no query sees them: page tails, pages of no request, positions before the windows."""
    skip_unless(splits, 2 * new)
    b = Batch([(130, new), (40, new)], 4, 2, dim, 16, "NHD", 97 + dim)
    mask = dict(window=50, sinks=3)
    want = b.want(**mask, gathered=splits == "gather")
    clean = b.device()
    seen = np.zeros(b.cache.codes.shape[:1] + (16,), bool)
    for r, length in enumerate(b.lens):
        first = length - new
        for p in range(length):
            if p < 3 or p > first - 50:
                seen[b.table[r, p // 16], p % 16] = True
    codes = b.cache.codes.copy()
    b.cache.codes = np.where(seen[:, None, :, None, None], codes, 0xFF).astype(np.uint8)
    call = dict(clean, kv_cache=dev(b.cache.raw()))
    got = attend(kvq, call, splits, window=50, num_sinks=3)
    check(got, want)
    same = attend(kvq, clean, splits, window=50, num_sinks=3)
    assert np.array_equal(bits_of(got[0]), bits_of(same[0])) and torch.equal(got[1], same[1])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,splits", [(5, None), (70, None), (70, "gather")])
def test_later_tokens_nan_does_not_reach_earlier_rows(kvq, dim, new, splits):
    b = Batch([(40, new)], 4, 2, dim, 16, "NHD", 101 + dim)
    want = b.want(gathered=splits == "gather")
    p = 40 + new - 2                                                  # the last but one
    b.cache.codes[b.table[0, p // 16], :, p % 16] = 0x7F
    got = attend(kvq, b.device(), splits)
    out, lse = ref.bf16(bits_of(got[0])), got[1].cpu().numpy()
    assert np.all(np.abs(out[:new - 2] - want[0][:new - 2]) <= want[2][:new - 2])
    assert np.all(np.isfinite(lse[:new - 2])) and np.all(np.isnan(lse[new - 2:])) and np.all(np.isnan(out[new - 2:]))


@pytest.mark.parametrize("new,splits", [(1, None), (40, None), (40, "gather")])
def test_bad_pages_and_requests(kvq, new, splits):
    b = Batch([(100, new), (60, new), (50, new), (200, new)], 8, 2, 128, 16, "HND", 103)
    b.table[0, 2] = -1
    b.table[1, 1] = b.cache.codes.shape[0]
    b.table = b.table[:, :10].copy()                                  # request 3 goes past the table
    want = b.want(gathered=splits == "gather")
    call = b.device()
    call["query_start"][3] += new + 1                                 # 2: too many tokens, 3: a negative range
    out = bf16_dev(np.full(b.q_bits.shape, CANARY, np.uint16))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = attend(kvq, dict(call, out=out, status=status), splits)
    check(got, want, 2 * new)
    assert np.all(bits_of(out)[2 * new:] == CANARY)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX | kvq.STATUS_BAD_BATCH
    call = b.device()
    status.zero_()
    check(attend(kvq, dict(call, status=status), splits), want)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX


@pytest.mark.parametrize("window", [0, 120])
def test_sequences_past_the_workspace_are_skipped(kvq, window):
    """max_seq_len has to hold where entries are gathered: a longer sequence's rows stay as they are."""
    b = Batch([(60, 40), (300, 40), (20, 40)], 8, 2, 128, 16, "NHD", 104)
    call = dict(b.device(), max_seq_len=128)
    out = bf16_dev(np.full(b.q_bits.shape, CANARY, np.uint16))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = attend(kvq, dict(call, out=out, status=status), "gather", window=window)
    want = b.want(gathered=True, window=window)
    keep = np.r_[0:40, 80:120]
    o = ref.bf16(bits_of(got[0]))
    assert np.all(np.abs(o[keep] - want[0][keep]) <= want[2][keep])
    skipped = np.all(bits_of(out)[40:80] == CANARY)
    assert skipped == (int(status.item()) == kvq.STATUS_BAD_BATCH) and skipped


@pytest.mark.parametrize("new", [2, 90])
def test_strides_and_extreme_queries(kvq, new):
    """Queries and outputs as slices of wider rows; rows of zeros, of the largest and of the smallest values."""
    b = Batch([(60, new), (33, new)], 6, 2, 64, 16, "NHD", 107)
    b.q_bits[0] = 0
    b.q_bits[1, 0] = ref.to_bf16(np.full(64, 1e-38))
    b.q_bits[1, 1] = ref.to_bf16(np.full(64, 3e30))
    b.q_bits[1, 1, 1:] = ref.to_bf16(np.full(63, 1e-30))
    b.scale = 1e-31
    call = b.device()
    T = b.q_bits.shape[0]
    wide = torch.zeros((T, 10, 64), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:8] = call["q"]
    outs = torch.zeros((T, 9, 64), dtype=torch.bfloat16, device=DEV)
    lses = torch.zeros((T, 11), device=DEV)
    got = attend(kvq, dict(call, q=wide[:, 2:8], out=outs[:, 1:7], lse=lses[:, 3:9]), None)
    check(got, b.want())
    assert bool((outs[:, 0] == 0).all()) and bool((outs[:, 7:] == 0).all()) and bool((lses[:, :3] == 0).all())
    for scale in (0.0, -0.125):
        b.scale = scale
        b.q_bits[1, 1] = b.q_bits[2, 1]
        check(attend(kvq, b.device(), None, window=20), b.want(window=20))
        if new > 48:
            check(attend(kvq, b.device(), "gather", window=20), b.want(window=20, gathered=True))


@pytest.mark.parametrize("new", [1, 64])
def test_offsets_past_32_bits(kvq, new):
    """Pages beyond the first 4 GB of the cache."""
    block, kv, dim = 64, 8, 128
    pages = (1 << 32) // (2 * block * kv * dim) + 40
    b = Batch([(150, new)], 8, kv, dim, block, "NHD", 109)
    raw = torch.zeros((pages, 2, block, kv, dim), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((pages, 2, kv), dtype=torch.uint8, device=DEV)
    call = b.device()
    want, gathered = b.want(), b.want(gathered=True)
    used = b.table[0][b.table[0] >= 0]
    moved = {int(p): pages - 1 - 3 * i for i, p in enumerate(used)}
    for p, to in moved.items():
        raw[to], scales[to] = call["kv_cache"][p], call["kv_scales"][p]
    b.table = np.array([[moved.get(int(p), -1) for p in b.table[0]]])
    call = dict(call, kv_cache=raw, kv_scales=scales, block_table=dev(b.table.astype(np.int32)))
    check(attend(kvq, call, None), want)
    if new > 48:
        check(attend(kvq, call, "gather"), gathered)
    # and appended there
    key = torch.randn((new, kv, dim), device=DEV).to(torch.bfloat16)
    kvq.kvq_rope_append_fp8_per_head(None, key, key, torch.zeros(new, dtype=torch.int64, device=DEV),
                                     torch.cat([torch.ones((1, 8)), torch.zeros((1, 8))], 1).to(DEV), i32([0, new]),
                                     i32([150 + new]), call["block_table"], raw, scales, new)
    p = 150 + new - 1
    page = int(b.table[0, p // block])
    e = scales[page, 1].float() - 127
    back = raw[page, 1, p % block].view(torch.float8_e4m3fn).float() * torch.exp2(e)[:, None]
    assert bool(((back - key[-1].float()).abs() <= 2.0 ** -4 * key[-1].float().abs() + 2.0 ** -10 * torch.exp2(e)[:, None]).all())


@pytest.mark.parametrize("dim,new", [(64, 1), (128, 1), (256, 1), (128, 8), (128, 80)])
def test_long_sequences_with_default_splits(kvq, dim, new):
    b = Batch([(5000, new), (17, new), (2900, new)], 8, 2, dim, 64, "NHD", 113)
    check(attend(kvq, b.device(), None), b.want())


@pytest.mark.parametrize("dim,layout", [(64, "HND"), (128, "NHD"), (256, "NHD")])
@pytest.mark.parametrize("new", [1, 2, 20, 40])
@pytest.mark.parametrize("splits", [1, -2, "gather"])
def test_rows_whose_maximum_grows(kvq, dim, layout, new, splits):
    """Scores that rise along the keys, past every reference, and fall again."""
    skip_unless(splits, 2 * new)
    b = Batch([(450, new), (200, new)], 4, 2, dim, 16, layout, 127 + dim + new)
    for r, length in enumerate(b.lens):
        for col in range(-(-length // 16)):
            b.cache.scales[b.table[r, col], 0] = 127 - 16 + min(col // 2, 9)
    check(attend(kvq, b.device(), splits), b.want(gathered=splits == "gather"))


@pytest.mark.parametrize("dim,heads,kv,new", [(64, 6, 2, 11), (64, 6, 2, 21), (64, 6, 2, 22), (128, 8, 2, 8), (128, 8, 2, 9),
                                              (256, 8, 2, 4), (256, 8, 2, 5), (128, 14, 2, 4)])
@pytest.mark.parametrize("splits", [1, -2, None])
def test_rows_on_both_sides_of_the_kernels_limits(kvq, dim, heads, kv, new, splits):
    b = Batch([(300, new), (77, new)], heads, kv, dim, 16, "NHD", 131)
    check(attend(kvq, b.device(), splits), b.want())


@pytest.mark.parametrize("dim,heads,kv,new", [(64, 8, 2, 3), (128, 8, 2, 3), (128, 14, 2, 4), (256, 8, 2, 3)])
def test_many_requests_of_a_few_rows(kvq, dim, heads, kv, new):
    """Enough requests that blocks of 16 rows fill the GPU."""
    b = Batch([(int(c), new) for c in np.random.default_rng(5).integers(0, 40, 300)], heads, kv, dim, 16, "NHD", 137)
    check(attend(kvq, b.device(), None), b.want())


@pytest.mark.parametrize("at_once", [1, 31, 32, 33, 70])
def test_gathering_many_requests(kvq, at_once):
    """More and fewer requests at a time than are put in order of their lengths, equal lengths and none among them."""
    rng = np.random.default_rng(151)
    reqs = [(int(c), int(n)) for c, n in zip(rng.choice([0, 5, 5, 64, 200, 333], 70), rng.choice([0, 1, 13, 30, 30], 70))]
    reqs[3] = (17, 30)
    b = Batch(reqs, 4, 2, 64, 16, "HND", 151)
    call = b.device()
    for mask in ({}, dict(window=40, num_sinks=3)):
        got = kvq.kvq_window_attention_fp8_per_head(**gathering(kvq, call, at_once, **mask), **mask)
        check(got, b.want(gathered=True, window=mask.get("window", 0), sinks=mask.get("num_sinks", 0)))


@pytest.mark.parametrize("new,splits", [(1, 4), (1, -4), (1, 1), (40, 1), (40, -3), (40, "gather")])
def test_graphs_and_streams(kvq, new, splits):
    b = Batch([(300, new), (90, new)], 8, 2, 128, 16, "NHD", 139)
    call = b.device()
    want = attend(kvq, call, splits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attend(kvq, dict(call, stream=side), splits)
    torch.cuda.synchronize()
    assert np.array_equal(bits_of(got[0]), bits_of(want[0])) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = attend(kvq, call, splits)
    call["q"].copy_(call["q"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    again = attend(kvq, call, splits)
    assert np.array_equal(bits_of(inside[0]), bits_of(again[0])) and torch.equal(inside[1], again[1])


def test_attention_refuses_what_does_not_fit(kvq):
    call = Batch([(30, 1)], 4, 2, 64, 16, "NHD", 149).device()

    def refused(kind, match, **over):
        with pytest.raises(kind, match=match):
            kvq.kvq_window_attention_fp8_per_head(**{**call, **over})

    refused(ValueError, "kv_scales", kv_scales=None)
    refused(ValueError, "kv_scales", kv_scales=call["kv_scales"].float())
    refused(ValueError, "kv_scales", kv_scales=call["kv_scales"][:-1])
    refused(ValueError, "kv_scales", kv_scales=call["kv_scales"].transpose(0, 1).contiguous().transpose(0, 1))
    refused(ValueError, "kv_scales", kv_scales=call["kv_scales"].cpu())
    refused(ValueError, "kv_cache", kv_cache=call["kv_cache"][..., :32])
    refused(ValueError, "kv_cache", kv_cache=call["kv_cache"].float())
    refused(ValueError, "kv_cache", layout="HND", kv_cache=call["kv_cache"][:, :, :, :1])
    refused(ValueError, "layout", layout="XYZ")
    refused(ValueError, "q", q=call["q"].float())
    refused(ValueError, "seq_lens", seq_lens=call["seq_lens"].long())
    refused(ValueError, "query_start", query_start=call["query_start"][:1])
    refused(RuntimeError, "num_heads", q=call["q"][:, :3])
    refused(RuntimeError, "num_splits", num_splits=129)
    refused(RuntimeError, "softmax_scale", softmax_scale=float("nan"))
    refused(RuntimeError, "num_sinks", num_sinks=-1)


@pytest.mark.parametrize("dim,heads,kv", [(64, 8, 2), (128, 8, 2), (256, 4, 1)])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 100, 40])
@pytest.mark.parametrize("splits", [1, -5, "gather"])
def test_padded_requests_and_windows_of_any_size(kvq, dim, heads, kv, window, splits):
    """Queries at negative positions beside others of their request, under windows that reach past the first position
    by any amount: as if there were none, or the window of the others."""
    b = Batch([(0, 130), (20, 130), (0, 130), (90, 130)], heads, kv, dim, 16, "NHD", 157)
    b.lens[0], b.lens[2] = 80, 5                                      # their first 50 and 125 positions are negative
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = attend(kvq, b.device(), splits, window=window, num_sinks=3, status=status)
    check(got, b.want(window=window, sinks=3))
    assert int(status.item()) == 0
    if window > 1000:
        whole = attend(kvq, b.device(), splits)
        assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])


def spare_bytes(call):
    """The call's results, and the most memory that it held beside what was there before."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = call()
    torch.cuda.synchronize()
    return got, torch.cuda.max_memory_allocated() - before


def widened(call, columns):
    """The call with a block table of so many columns."""
    table = torch.zeros((call["block_table"].shape[0], columns), dtype=torch.int32, device=DEV)
    table[:, :call["block_table"].shape[1]] = call["block_table"]
    return dict(call, block_table=table)


def test_default_room_for_gathered_entries(kvq):
    """A batch whose entries take more than 1 GiB for the bound on its lengths goes through in rounds within it; where
    not one request's fit they are decoded as they are read."""
    b = Batch([(300, 640), (0, 640), (77, 640)], 64, 8, 128, 64, "NHD", 163)
    call, results = widened(b.device(), (1 << 20) // 64), 1920 * 64 * (2 * 128 + 4)
    room = kvq.kvq_fp8_attention_workspace_bytes(1920, 64, 8, 128, 3, 640, 1000)
    want = kvq.kvq_window_attention_fp8_per_head(**dict(call, max_seq_len=1000), num_splits=1,
                                                 workspace=torch.empty(room, dtype=torch.uint8, device=DEV))
    assert kvq.kvq_fp8_attention_default_splits(640, 64, 8, 128, 3, 131072) == (1, True)      # one request at a time
    got, held = spare_bytes(lambda: attend(kvq, dict(call, max_seq_len=131072), None))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert results < held <= results + (1 << 30) + (1 << 22)
    splits, through = kvq.kvq_fp8_attention_default_splits(640, 64, 8, 128, 3, 1 << 20)       # 4 GiB a request
    assert splits > 1 or not through
    call = dict(call, max_seq_len=1 << 20)
    want = attend(kvq, call, -splits if through else splits)
    got, held = spare_bytes(lambda: attend(kvq, call, None))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and held < results + (1 << 29)


def test_a_larger_workspace_of_ones_own(kvq):
    """With room given for every entry the default gathers, however much that takes."""
    b = Batch([(10 * i, 128) for i in range(16)], 32, 8, 128, 64, "NHD", 173)
    call = dict(widened(b.device(), 40000 // 64), max_seq_len=40000)
    splits, through = kvq.kvq_fp8_attention_default_splits(128, 32, 8, 128, 16, 40000)
    assert splits > 1 or not through
    room = kvq.kvq_fp8_attention_workspace_bytes(2048, 32, 8, 128, 16, 128, 40000)
    assert room > 1 << 31
    held = torch.empty(room, dtype=torch.uint8, device=DEV)
    want = kvq.kvq_window_attention_fp8_per_head(**call, num_splits=1, workspace=held)
    held.fill_(0xFF)
    got = kvq.kvq_window_attention_fp8_per_head(**call, workspace=held)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not bool((held[:128 * 8 * 128 * 2] == 0xFF).all())         # (the first request's entries are there)


@pytest.mark.parametrize("dim,heads,kv,new,layout", [(64, 64, 8, 130, "NHD"), (128, 32, 8, 300, "HND"), (256, 32, 4, 130, "NHD")])
@pytest.mark.parametrize("mask", [dict(), dict(window=400, num_sinks=5)])
def test_default_calls_attend_sequences_of_any_length(kvq, dim, heads, kv, new, layout, mask):
    """A bound on the lengths that does not hold, for one request, for all but one, and in a captured call whose
    sequences grow: every row is as for a bound that does, or as where its entries are decoded as they are read."""
    b = Batch([(100, new), (900, new), (0, new), (700, 7), (30, 0), (3, 1)], heads, kv, dim, 16, layout, 179)
    call = b.device()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gathered, read = attend(kvq, call, "gather", **mask), attend(kvq, call, 1, **mask)
    for bound in (500, new + 1, 1, 0):
        through = kvq.kvq_fp8_attention_default_splits(new, heads, kv, dim, 6, bound, *mask.values())
        assert through == (1, bound > 0)                              # (a bound of 0 makes no call: not gathered)
        got = attend(kvq, dict(call, max_seq_len=bound, status=status), None, **mask)
        rows = kvq.kvq_fp8_attention_workspace_bytes(b.start[-1], heads, kv, dim, 1, new, bound, *mask.values()) // (
            4 * kv * dim) // 64 * 64 if bound else -1
        for r, length in enumerate(b.lens):
            first = max(0, length - b.reqs[r][1] - 399) if mask else 0
            want = gathered if length - first + min(mask.get("num_sinks", 0), first) <= rows else read
            t = slice(b.start[r], b.start[r + 1])
            assert torch.equal(got[0][t], want[0][t]) and torch.equal(got[1][t], want[1][t]), (bound, r)
        assert int(status.item()) == 0
    lens = call["seq_lens"].clone()
    call["seq_lens"].copy_(torch.clamp(lens, max=new + 50))
    short = dict(call, max_seq_len=new + 50)
    attend(kvq, short, None, **mask)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = attend(kvq, short, None, **mask)
    call["seq_lens"].copy_(lens)
    graph.replay()
    torch.cuda.synchronize()
    again = attend(kvq, short, None, **mask)
    assert torch.equal(inside[0], again[0]) and torch.equal(inside[1], again[1])
    assert bool(torch.isfinite(inside[1]).all())
    # requests that are none are reported once more, and their rows left
    call["query_start"][4] = b.start[-1] + 1
    out = bf16_dev(np.full(b.q_bits.shape, CANARY, np.uint16))
    attend(kvq, dict(call, max_seq_len=500, out=out, status=status), None, **mask)
    assert int(status.item()) == kvq.STATUS_BAD_BATCH
    left = np.all(bits_of(out) == CANARY, (1, 2))
    assert np.all(left[b.start[3]:b.start[5]]) and not np.any(left[:b.start[3]]) and not np.any(left[b.start[5]:])


@pytest.mark.parametrize("splits", [1, -3, "gather", None])
@pytest.mark.parametrize("mask", [dict(), dict(window=90, num_sinks=4)])
def test_sequences_of_the_largest_lengths(kvq, splits, mask):
    """Lengths next to 2^31, far past the block table: the keys that it holds are attended to, or none where the window
    lies behind them but for the first."""
    b = Batch([(200, 70), (50, 70), (90, 70)], 16, 8, 64, 16, "NHD", 181)
    b.table = b.table[:, :9].copy()                                   # 144 positions
    lens = [(1 << 31) - 1, 120, (1 << 31) - 70]
    call = dict(b.device(), seq_lens=i32(lens))
    b.table[b.table < 0] = b.cache.codes.shape[0]
    call["block_table"] = dev(b.table.astype(np.int32))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = attend(kvq, dict(call, status=status), splits, **mask)
    assert int(status.item()) == kvq.STATUS_BAD_INDEX
    # every query of theirs is past the table: it sees all of it, or the first keys alone
    b.lens = [144 + 70, 120, 144 + 70]
    if mask:
        b.lens = [144 + 1000, 120, 144 + 1000]
    check(got, b.want(window=mask.get("window", 0), sinks=mask.get("num_sinks", 0)))


@pytest.mark.parametrize("dim,heads,kv", [(64, 32, 4), (128, 32, 8), (256, 16, 4)])
def test_a_chunk_beside_decoded_tokens(kvq, dim, heads, kv):
    """One request's chunk and the decoded tokens of many in one call, appended and attended to as by default."""
    reqs = [(int(c), 1) for c in np.random.default_rng(7).integers(0, 300, 40)]
    reqs[17:17] = [(150, 400), (0, 33)]
    b = Batch(reqs, heads, kv, dim, 16, "NHD", 191)
    case = Append(reqs, heads, kv, dim, 16, "NHD", dim, 193)
    check_append(kvq, case)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert kvq.kvq_fp8_attention_default_splits(400, heads, kv, dim, 42, max(b.lens)) == (1, True)
    check(attend(kvq, dict(b.device(), status=status), None), b.want(gathered=True))
    assert int(status.item()) == 0


def test_defaults_for_sizes_that_make_no_call(kvq):
    most = (1 << 31) - 1
    for args in ((300, 32, 8, 0, 64, 6000), (300, 32, 8, -128, 64, 6000), (most, most, 1, 128, most, most),
                 (1 << 20, 1 << 20, 1 << 20, 128, 1 << 20, 6000), (300, 32, 8, 128, 65536, 6000)):
        assert kvq.kvq_fp8_attention_default_splits(*args) == (1, False)
        assert kvq.kvq_per_head_attention_default_splits(*args) == (1, False)
