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

    def run(self, kvq, status=None, in_place=False, no_q=False, no_k=False, stream=None, cos_sin=None):
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
            i32(self.start), i32(self.lens), dev(self.table.astype(np.int32)), cache, scales, max([n for _, n in self.reqs] + [0]),
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
