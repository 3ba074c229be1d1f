"""Serving from the per-head e4m3 cache and attention over whole prompts
without a GPU: the entry points refuse bad arguments on the host before any
CUDA call, the Python calls refuse tensors of the wrong kind, and the plain
reference's number formats.  Nothing is launched; the tests that pass fake
device addresses are skipped where a GPU is visible."""
import numpy as np
import pytest
import torch

import fp8_per_head_reference as ref

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-pointer validation tests run only on GPU-less hosts")

A = 0x10000000          # a 256-byte-aligned fake device address, never dereferenced


@pytest.fixture(scope="module")
def kvq():
    from fp8_quantized_paged_concat_gb300 import _build
    _build.build()
    import fp8_quantized_paged_concat_gb300 as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def lib(kvq):
    return kvq.load_library()


def rejected(lib, name, args, needle):
    assert getattr(lib, name)(*args.values()) == 1
    text = lib.kvq_last_error_string().decode()
    assert needle in text and text.startswith(name + ":"), text


# --------------------------------------------------------------------------
# the reference's formats
# --------------------------------------------------------------------------

def test_reference_codes_are_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-14, 8, 20000), ref.MAGNITUDE, -ref.MAGNITUDE,
                        (ref.MAGNITUDE[1:] + ref.MAGNITUDE[:-1]) / 2, [0.0, -0.0, 448.0, -448.0]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.to_e4m3(x), want)
    assert ref.to_e4m3(np.float32([1e9, -np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7F]


def test_reference_exponent_is_the_least():
    assert ref.exponent(0.0) == -60 and ref.exponent(448.0) == 0 and ref.exponent(np.nextafter(448.0, 500)) == 1
    assert ref.exponent(3.5) == -7 and ref.exponent(3e38) == 60


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------

def append_args(**over):
    args = dict(q=A, q_stride_t=8 * 128, q_stride_h=128, k=A, k_stride_t=256, k_stride_h=128, v=A, v_stride_t=256,
                v_stride_h=128, positions=A, num_tokens=4, num_heads=8, num_kv_heads=2, head_size=128, cos_sin=A,
                cos_sin_stride=128, max_position=1000, rot_dim=128, interleaved=0, query_start=A, seq_lens=A, batch_size=4,
                max_query_len=1, block_table=A, block_table_stride=16, block_table_width=16, kv_cache=A, kv_scales=A,
                num_pages=64, block_size=16, layout=0, q_out=A, q_out_stride_t=8 * 128, q_out_stride_h=128, k_out=A,
                k_out_stride_t=256, k_out_stride_h=128, d_status=None, stream=None)
    assert set(over) <= set(args)
    return {**args, **over}


@no_gpu_only
@pytest.mark.parametrize("over,needle", [
    (dict(num_tokens=-1), "must be >= 0"),
    (dict(batch_size=-1), "must be >= 0"),
    (dict(max_query_len=-1), "must be >= 0"),
    (dict(head_size=96), "head_size must be 64, 128 or 256"),
    (dict(num_kv_heads=0), "must be positive"),
    (dict(num_heads=0), "must be positive"),
    (dict(rot_dim=24), "rot_dim"),
    (dict(rot_dim=144), "rot_dim"),
    (dict(num_tokens=1 << 31), "below 2^31"),
    (dict(max_query_len=1 << 27), "below 2^31"),
    (dict(layout=2), "layout"),
    (dict(kv_cache=None), "kv_cache must be non-NULL"),
    (dict(kv_cache=A + 8), "16-byte aligned"),
    (dict(kv_scales=None), "kv_scales must be non-NULL"),
    (dict(num_pages=0), "num_pages"),
    (dict(block_size=0), "block_size positive"),
    (dict(block_size=1 << 24), "below 2^31"),
    (dict(q=A + 8), "q must be non-NULL and 16-byte aligned"),
    (dict(q_out=None), "q_out must be non-NULL"),
    (dict(q_out_stride_t=1016), "rows must not overlap"),
    (dict(k=None), "k must be non-NULL"),
    (dict(v=None), "v must be non-NULL"),
    (dict(k_stride_t=252), "k strides"),
    (dict(v_stride_h=120), "v strides"),
    (dict(k_out=A + 8), "k_out must be"),
    (dict(k_out_stride_t=128), "rows must not overlap"),
    (dict(positions=None), "bad positions"),
    (dict(max_position=0), "max_position"),
    (dict(cos_sin=None), "cos_sin"),
    (dict(cos_sin_stride=126), "cos_sin"),
    (dict(query_start=None), "non-NULL"),
    (dict(seq_lens=A + 1), "4-byte aligned"),
    (dict(batch_size=65536), "at most 65535"),
    (dict(block_table_width=0), "block_table_width"),
    (dict(block_table_stride=15), "block_table_stride"),
    (dict(d_status=A + 2), "d_status"),
])
def test_append_rejects_bad_arguments_on_host(lib, over, needle):
    rejected(lib, "kvq_rope_append_fp8_per_head", append_args(**over), needle)


@no_gpu_only
def test_append_of_nothing_is_ok_without_a_device(lib):
    for over in (dict(num_tokens=0), dict(batch_size=0), dict(max_query_len=0)):
        assert lib.kvq_rope_append_fp8_per_head(*append_args(**over).values()) == 0


def test_append_refuses_wrong_tensors(kvq):
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_rope_append_fp8_per_head(x, x, x, *[x] * 7, 1)
    with pytest.raises(ValueError, match="expected a tensor"):
        kvq.kvq_rope_append_fp8_per_head(x, None, x, *[x] * 7, 1)


# --------------------------------------------------------------------------
# attention over the cache
# --------------------------------------------------------------------------

INT_MAX = (1 << 31) - 1


def window_args(**over):
    args = dict(q=A, q_stride_t=8 * 128, q_stride_h=128, num_tokens=4, num_heads=8, query_start=A, seq_lens=A,
                batch_size=4, max_query_len=1, block_table=A, block_table_stride=16, block_table_width=16, kv_cache=A,
                kv_scales=A, num_pages=64, block_size=16, layout=0, num_kv_heads=2, head_size=128, softmax_scale=0.1,
                window=0, num_sinks=0, out=A, out_stride_t=8 * 128, out_stride_h=128, lse=A, lse_stride_t=8,
                max_seq_len=256, num_splits=1, workspace=None, workspace_bytes=0, d_status=None, stream=None)
    assert set(over) <= set(args)
    return {**args, **over}


# 40 query rows per key head, and the least workspace for one request's 256 entries
ROWS = dict(num_tokens=40, max_query_len=10)
HELD = 256 * 2 * 128 * 4 + 48


@no_gpu_only
@pytest.mark.parametrize("over,needle", [
    (dict(num_tokens=-1), "must be >= 0"),
    (dict(max_seq_len=-1), "must be >= 0"),
    (dict(num_splits=0), "num_splits"),
    (dict(num_splits=129), "num_splits"),
    (dict(num_sinks=-1), "num_sinks"),
    (dict(head_size=96), "head_size must be 64, 128 or 256"),
    (dict(num_heads=7), "num_heads must be a positive multiple"),
    (dict(num_kv_heads=0), "num_heads must be a positive multiple"),
    (dict(max_query_len=1 << 28), "below 2^31"),
    (dict(kv_cache=None), "kv_cache must be non-NULL"),
    (dict(kv_cache=A + 8), "16-byte aligned"),
    (dict(kv_scales=None), "kv_scales must be non-NULL"),
    (dict(num_pages=0), "num_pages"),
    (dict(num_pages=1 << 31), "num_pages"),
    (dict(block_size=0), "block_size positive"),
    (dict(layout=2), "layout"),
    (dict(q=A + 8), "q must be"),
    (dict(q_stride_t=1028), "q strides"),
    (dict(out=None), "out must be"),
    (dict(out_stride_t=1016), "rows must not overlap"),
    (dict(lse=A + 2), "lse"),
    (dict(lse_stride_t=7), "lse"),
    (dict(query_start=None), "non-NULL"),
    (dict(batch_size=65536), "at most 65535"),
    (dict(block_table_width=0), "block_table_width"),
    (dict(block_table_stride=15), "block_table_stride"),
    (dict(block_table_width=1 << 27, block_table_stride=1 << 27), "block_table_width * block_size"),
    (dict(softmax_scale=float("inf")), "softmax_scale must be finite"),
    (dict(softmax_scale=2.4e38), "softmax_scale must be finite"),
    (dict(num_splits=16), "workspace must be non-NULL"),
    (dict(num_splits=2, **ROWS), "workspace must be non-NULL"),
    (dict(workspace=A, workspace_bytes=HELD - 1, **ROWS), "workspace must be 16-byte aligned"),
    (dict(workspace=A + 8, workspace_bytes=HELD + 64, **ROWS), "workspace must be 16-byte aligned"),
    (dict(d_status=A + 2), "d_status"),
])
def test_attention_rejects_bad_arguments_on_host(lib, over, needle):
    rejected(lib, "kvq_window_attention_fp8_per_head", window_args(**over), needle)


@no_gpu_only
@pytest.mark.parametrize("over", [{}, dict(num_splits=8), dict(window=-5, num_sinks=INT_MAX, max_seq_len=INT_MAX),
                                  dict(lse=None, lse_stride_t=0), dict(q_stride_t=0), dict(max_seq_len=0),
                                  dict(workspace=A, workspace_bytes=0),                       # few rows: not looked at
                                  dict(workspace=A, workspace_bytes=HELD, **ROWS),
                                  dict(workspace=A, workspace_bytes=HELD, max_seq_len=INT_MAX, **ROWS),   # the table's reach
                                  dict(workspace=A, workspace_bytes=0, q_stride_t=0, **ROWS)])            # decoded all the same
def test_attention_accepts_good_arguments(lib, over):
    """Without a device the first thing that fails is the device query."""
    assert lib.kvq_window_attention_fp8_per_head(*window_args(**over).values()) in (2, 3), lib.kvq_last_error_string()


@no_gpu_only
@pytest.mark.parametrize("over", [dict(num_tokens=0), dict(batch_size=0), dict(max_query_len=0)])
def test_attention_of_nothing_is_ok_without_a_device(lib, over):
    nothing = dict(q=None, out=None, kv_cache=None, kv_scales=None, block_table=None, query_start=None, seq_lens=None)
    assert lib.kvq_window_attention_fp8_per_head(*window_args(**over, **nothing).values()) == 0


@no_gpu_only
def test_attention_of_any_length_checks_as_the_other_does(lib):
    name = "kvq_window_attention_fp8_per_head_any_length"
    for over, needle in ((dict(num_splits=0), "num_splits"), (dict(kv_scales=None), "kv_scales must be non-NULL"),
                         (dict(workspace=A, workspace_bytes=HELD - 1, **ROWS), "workspace must be 16-byte aligned"),
                         (dict(softmax_scale=float("inf")), "softmax_scale must be finite")):
        rejected(lib, name, window_args(**over), needle)
    for over in ({}, dict(workspace=A, workspace_bytes=HELD, **ROWS), dict(max_seq_len=0)):
        assert getattr(lib, name)(*window_args(**over).values()) in (2, 3), lib.kvq_last_error_string()
    nothing = dict(q=None, out=None, kv_cache=None, kv_scales=None, block_table=None, query_start=None, seq_lens=None)
    assert getattr(lib, name)(*window_args(num_tokens=0, **nothing).values()) == 0


@pytest.mark.parametrize("args,want", [
    ((40, 8, 2, 128, 1, 10, 256, 0, 0, 1), HELD),
    ((40, 8, 2, 128, 4, 10, 200, 0, 0, 1), 4 * 256 * 2 * 128 * 4 + (4 * 8 + 3 + 3) // 4 * 16),
    ((40, 8, 2, 128, 1, 10, 5000, 100, 20, 1), 192 * 2 * 128 * 4 + 48),               # 100 + 9 + 20 keys
    ((40, 8, 2, 128, 1, 10, 0, 0, 0, 1), 64 * 2 * 128 * 4 + 32),
    ((4, 8, 2, 128, 4, 1, 256, 0, 0, 1), 0),
    ((4, 8, 2, 128, 4, 1, 256, 0, 0, 16), 4 * 8 * 129 * 4 * 16),
    ((0, 8, 2, 128, 1, 10, 256, 0, 0, 1), -1), ((40, 8, 0, 128, 1, 10, 256, 0, 0, 1), -1),
    ((40, 1, 2, 128, 1, 10, 256, 0, 0, 1), -1), ((40, 8, 2, 0, 1, 10, 256, 0, 0, 1), -1),
    ((40, 8, 2, 128, 0, 10, 256, 0, 0, 1), -1), ((40, 8, 2, 128, 1, 0, 256, 0, 0, 1), -1),
    ((40, 8, 2, 128, 1, 10, -1, 0, 0, 1), -1), ((40, 8, 2, 128, 1, 10, 256, 0, -1, 1), -1),
    ((40, 8, 2, 128, 1, 10, 256, 0, 0, 0), -1),
    ((40, INT_MAX, INT_MAX, INT_MAX, INT_MAX, 64, INT_MAX, 0, 0, 1), -1),
])
def test_attention_workspace_bytes(lib, args, want):
    assert lib.kvq_fp8_attention_workspace_bytes(*args) == want


@no_gpu_only
def test_default_splits_without_a_device(kvq):
    assert kvq.kvq_fp8_attention_default_splits(1, 8, 2, 128, 1, 4096) == (1, False)
    assert kvq.kvq_fp8_attention_default_splits(0, 8, 0, 128, 0, 0) == (1, False)


def test_attention_refuses_wrong_tensors(kvq):
    bf = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    cache, scales = torch.zeros((4, 2, 16, 2, 128), dtype=torch.uint8), torch.zeros((4, 2, 2), dtype=torch.uint8)
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        kvq.kvq_window_attention_fp8_per_head(bf, ints, ints, ints, cache, scales, 1.0, 1, 1)
    with pytest.raises(ValueError, match="q: expected a tensor"):
        kvq.kvq_window_attention_fp8_per_head([1.0], ints, ints, ints, cache, scales, 1.0, 1, 1)


# --------------------------------------------------------------------------
# attention over whole prompts
# --------------------------------------------------------------------------

def prompt_args(**over):
    args = dict(q=A, q_stride_t=8 * 128, q_stride_h=128, k=A, k_stride_t=256, k_stride_h=128, v=A, v_stride_t=256,
                v_stride_h=128, num_tokens=40, num_heads=8, num_kv_heads=2, head_size=128, seq_start=A, batch_size=4,
                max_seq_len=40, softmax_scale=0.1, window=0, num_sinks=0, out=A, out_stride_t=8 * 128, out_stride_h=128,
                lse=A, lse_stride_t=8, d_status=None, stream=None)
    assert set(over) <= set(args)
    return {**args, **over}


@no_gpu_only
@pytest.mark.parametrize("over,needle", [
    (dict(num_tokens=-1), "must be >= 0"),
    (dict(batch_size=-1), "must be >= 0"),
    (dict(max_seq_len=-1), "must be >= 0"),
    (dict(num_sinks=-1), "num_sinks"),
    (dict(head_size=96), "head_size must be 64, 128 or 256"),
    (dict(head_size=512), "head_size must be 64, 128 or 256"),
    (dict(num_heads=7), "num_heads must be a positive multiple"),
    (dict(num_heads=0), "num_heads must be a positive multiple"),
    (dict(num_kv_heads=0), "num_heads must be a positive multiple"),
    (dict(batch_size=65536), "at most 65535"),
    (dict(num_tokens=1 << 28), "below 2^31"),
    (dict(num_tokens=(1 << 28) - 16000), "below 2^31"),
    (dict(q=A + 8), "q must be"),
    (dict(k=None), "k must be"),
    (dict(v=A + 4), "v must be"),
    (dict(k_stride_t=252), "k strides"),
    (dict(q_stride_t=0), "strides must be positive"),
    (dict(k_stride_h=0), "k strides"),
    (dict(v_stride_t=-256), "strides"),
    (dict(v_stride_t=1 << 38), "strides must be positive and below 2^38"),
    (dict(out=None), "out must be"),
    (dict(out_stride_t=1016), "rows must not overlap"),
    (dict(lse=A + 2), "lse"),
    (dict(lse_stride_t=7), "lse"),
    (dict(seq_start=None), "seq_start"),
    (dict(seq_start=A + 2), "seq_start"),
    (dict(softmax_scale=float("nan")), "softmax_scale must be finite"),
    (dict(softmax_scale=-2.4e38), "softmax_scale must be finite"),
    (dict(d_status=A + 2), "d_status"),
])
def test_prompt_attention_rejects_bad_arguments_on_host(lib, over, needle):
    rejected(lib, "kvq_prompt_attention", prompt_args(**over), needle)


@no_gpu_only
@pytest.mark.parametrize("over", [{}, dict(window=-5, num_sinks=INT_MAX, max_seq_len=INT_MAX), dict(lse=None, lse_stride_t=0),
                                  dict(num_heads=300, num_kv_heads=1, q_stride_t=300 * 128, out_stride_t=300 * 128,
                                       lse_stride_t=300)])
def test_prompt_attention_accepts_good_arguments(lib, over):
    """Without a device the first thing that fails is the device query."""
    assert lib.kvq_prompt_attention(*prompt_args(**over).values()) in (2, 3), lib.kvq_last_error_string()


@no_gpu_only
@pytest.mark.parametrize("over", [dict(num_tokens=0), dict(batch_size=0), dict(max_seq_len=0)])
def test_prompt_attention_of_nothing_is_ok_without_a_device(lib, over):
    nothing = dict(q=None, k=None, v=None, out=None, seq_start=None)
    assert lib.kvq_prompt_attention(*prompt_args(**over, **nothing).values()) == 0


def test_prompt_attention_refuses_wrong_tensors(kvq):
    bf = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        kvq.kvq_prompt_attention(bf, bf, bf, torch.zeros(2, dtype=torch.int32), 1.0, 2)
    with pytest.raises(ValueError, match="q: expected a tensor"):
        kvq.kvq_prompt_attention(None, bf, bf, torch.zeros(2, dtype=torch.int32), 1.0, 2)
