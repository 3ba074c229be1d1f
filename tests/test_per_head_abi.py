"""Serving from the per-head NVFP4 cache without a GPU: the four entry points
refuse bad arguments on the host before any CUDA call, the Python calls refuse
tensors of the wrong kind, sizes and bounds of the helpers, and the plain
reference's number formats.  Nothing is launched; the tests that pass fake
device addresses are skipped where a GPU is visible."""
import numpy as np
import pytest
import torch

import per_head_reference as ref

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-pointer validation tests run only on GPU-less hosts")

A = 0x10000000          # a 256-byte-aligned fake device address, never dereferenced
INT_MAX = 2 ** 31 - 1


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


def err(lib):
    return lib.kvq_last_error_string().decode()


def rejected(lib, name, args, needle):
    assert getattr(lib, name)(*args.values()) == 1
    assert needle in err(lib), err(lib)
    assert err(lib).startswith(name + ":")


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------

def window_args(**over):
    args = dict(q=A, q_stride_t=8 * 128, q_stride_h=128, num_tokens=4, num_heads=8, query_start=A, seq_lens=A,
                batch_size=4, max_query_len=1, block_table=A, block_table_stride=16, block_table_width=16, kv_cache=A,
                num_pages=64, block_size=16, layout=0, num_kv_heads=2, head_size=128, k_scale=A, v_scale=A,
                softmax_scale=0.1, window=0, num_sinks=0, out=A, out_stride_t=8 * 128, out_stride_h=128, lse=A,
                lse_stride_t=8, max_seq_len=256, num_splits=1, workspace=None, workspace_bytes=0, d_status=None,
                stream=None)
    assert set(over) <= set(args)
    return {**args, **over}


def tree_args(**over):
    w = window_args(**{k: v for k, v in over.items() if k in window_args()})
    out = {}
    for k, v in w.items():
        if k in ("window", "num_sinks"):
            continue
        if k == "block_table":
            out.update(tree_mask=A, tree_mask_stride=1, mask_words=1)
        out[k] = v
    return {**out, **over}


ATTENTION_REFUSALS = [
    (dict(num_tokens=-1), "must be >= 0"),
    (dict(batch_size=-1), "must be >= 0"),
    (dict(max_query_len=-1), "must be >= 0"),
    (dict(max_seq_len=-1), "must be >= 0"),
    (dict(num_splits=0), "num_splits must be in [1, 128]"),
    (dict(num_splits=129), "num_splits must be in [1, 128]"),
    (dict(head_size=96), "head_size must be 64, 128 or 256"),
    (dict(num_kv_heads=0), "multiple of num_kv_heads"),
    (dict(num_kv_heads=3), "multiple of num_kv_heads"),
    (dict(num_heads=0), "multiple of num_kv_heads"),
    (dict(num_tokens=1 << 31), "below 2^31"),
    (dict(max_query_len=1 << 28), "below 2^31"),
    (dict(layout=2), "layout"),
    (dict(kv_cache=None), "kv_cache must be non-NULL"),
    (dict(kv_cache=A + 8), "kv_cache must be non-NULL and 16-byte aligned"),
    (dict(num_pages=0), "num_pages"),
    (dict(num_pages=1 << 31), "num_pages"),
    (dict(block_size=0), "block_size positive"),
    (dict(num_heads=1, num_kv_heads=1, block_size=1), "multiple of 16 below 2^31"),
    (dict(block_size=1 << 29), "below 2^31"),
    (dict(q=None), "q must be non-NULL"),
    (dict(q=A + 8), "q must be non-NULL and 16-byte aligned"),
    (dict(q_stride_t=1020), "q strides"),
    (dict(q_stride_t=-1024), "q strides"),
    (dict(q_stride_h=120), "q strides"),
    (dict(q_stride_h=132), "q strides"),
    (dict(q_stride_h=1 << 40), "q head stride too large"),
    (dict(out=None), "out must be non-NULL"),
    (dict(out_stride_t=1016), "rows must not overlap"),
    (dict(out_stride_t=0), "rows must not overlap"),
    (dict(lse=A + 2), "lse"),
    (dict(lse_stride_t=7), "lse"),
    (dict(batch_size=65536), "at most 65535"),
    (dict(query_start=None), "non-NULL"),
    (dict(seq_lens=None), "non-NULL"),
    (dict(block_table=None), "non-NULL"),
    (dict(seq_lens=A + 1), "4-byte aligned"),
    (dict(block_table_width=0), "block_table_width"),
    (dict(block_table_stride=15), "block_table_stride"),
    (dict(block_table_width=1 << 27, block_table_stride=1 << 27), "2^31 - 256"),
    (dict(k_scale=None), "k_scale"),
    (dict(v_scale=A + 2), "v_scale"),
    (dict(softmax_scale=float("nan")), "softmax_scale must be finite"),
    (dict(softmax_scale=float("inf")), "softmax_scale must be finite"),
    (dict(d_status=A + 2), "d_status"),
    (dict(num_splits=9), "workspace must be non-NULL"),                          # past a cluster's ranges
    (dict(num_splits=2, max_query_len=9), "workspace must be non-NULL"),         # 36 rows: no cluster
    (dict(num_splits=2, workspace=A, workspace_bytes=1), "workspace must be"),
    (dict(num_splits=2, workspace=A + 8, workspace_bytes=1 << 30), "16-byte aligned"),
]


@no_gpu_only
@pytest.mark.parametrize("over,needle", ATTENTION_REFUSALS + [(dict(num_sinks=-1), "num_sinks must be >= 0")])
def test_window_attention_rejects_bad_arguments_on_host(lib, over, needle):
    rejected(lib, "kvq_window_attention_nvfp4_per_head", window_args(**over), needle)


@no_gpu_only
@pytest.mark.parametrize("over,needle", ATTENTION_REFUSALS + [
    (dict(tree_mask=None), "tree_mask must be non-NULL"),
    (dict(tree_mask=A + 4), "tree_mask must be non-NULL, 8-byte aligned"),
    (dict(mask_words=0), "tree_mask"),
    (dict(mask_words=2), "tree_mask"),                                           # row stride 1
    (dict(max_query_len=65), "tree_mask"),                                       # 64 bits a row
])
def test_tree_attention_rejects_bad_arguments_on_host(lib, over, needle):
    rejected(lib, "kvq_tree_attention_nvfp4_per_head", tree_args(**over), needle)


@no_gpu_only
@pytest.mark.parametrize("over", [{}, dict(num_splits=8), dict(num_splits=8, max_query_len=8),
                                  dict(num_splits=128, workspace=A, workspace_bytes=4 * 8 * 128 * 129 * 4),
                                  dict(window=-5, num_sinks=INT_MAX, max_seq_len=INT_MAX), dict(lse=None, lse_stride_t=0),
                                  dict(q_stride_t=0), dict(window=INT_MAX, num_sinks=INT_MAX, num_splits=16, workspace=A,
                                                           workspace_bytes=1 << 30, max_seq_len=INT_MAX)])
def test_attention_accepts_good_arguments(lib, over):
    """Without a device the first thing that fails is the device query."""
    args = window_args(**over)
    assert lib.kvq_window_attention_nvfp4_per_head(*args.values()) in (2, 3), err(lib)


@no_gpu_only
@pytest.mark.parametrize("scale,good", [(2.35e38, True), (-2.35e38, True), (2.4e38, False), (-2.4e38, False), (2.99e38, False)])
def test_softmax_scales_that_overflow_in_base_two_are_refused(lib, scale, good):
    """The kernels' factor is softmax_scale * log2(e), in fp32: past 2.3586e38 it would be infinite."""
    assert (abs(np.float64(np.float32(scale)) * np.log2(np.e)) <= np.finfo(np.float32).max) == good
    for name, args in (("kvq_window_attention_nvfp4_per_head", window_args), ("kvq_tree_attention_nvfp4_per_head", tree_args)):
        if good:
            assert getattr(lib, name)(*args(softmax_scale=scale).values()) in (2, 3), err(lib)
        else:
            rejected(lib, name, args(softmax_scale=scale), "softmax_scale must be finite")


@no_gpu_only
@pytest.mark.parametrize("over", [dict(num_tokens=0), dict(batch_size=0), dict(max_query_len=0)])
def test_empty_calls_do_nothing(lib, over):
    """No rows: nothing else is looked at."""
    nothing = dict(q=None, out=None, kv_cache=None, block_table=None, query_start=None, seq_lens=None)
    assert lib.kvq_window_attention_nvfp4_per_head(*window_args(**over, **nothing).values()) == 0
    assert lib.kvq_tree_attention_nvfp4_per_head(*tree_args(**over, **nothing).values()) == 0


@pytest.mark.parametrize("args,want", [((1, 1, 64, 1), 65 * 4 + 12), ((4, 8, 128, 128), 4 * 8 * 128 * 129 * 4),
                                       ((0, 8, 128, 2), -1), ((4, 0, 128, 2), -1), ((4, 8, 0, 2), -1),
                                       ((4, 8, 128, 0), -1), ((4, 8, 128, -3), -1), ((1 << 62, 8, 128, 2), -1),
                                       ((1 << 40, INT_MAX, INT_MAX, INT_MAX), -1)])
def test_workspace_bytes(lib, args, want):
    assert lib.kvq_per_head_attention_workspace_bytes(*args) == want


@no_gpu_only
def test_default_splits_without_a_device(kvq):
    assert kvq.kvq_per_head_attention_default_splits(1, 8, 2, 128, 1, 4096) == (1, False)
    assert kvq.kvq_per_head_attention_default_splits(0, 8, 0, 128, 0, 0) == (1, False)


# --------------------------------------------------------------------------
# norm + rotation, compaction
# --------------------------------------------------------------------------

def norm_args(**over):
    args = dict(q=A, q_stride_t=1024, q_stride_h=128, k=A, k_stride_t=256, k_stride_h=128, q_weight=A, k_weight=A,
                positions=A, num_tokens=16, num_heads=8, num_kv_heads=2, head_size=128, cos_sin=A, cos_sin_stride=128,
                max_position=4096, rot_dim=128, interleaved=0, eps=1e-6, q_out=A, q_out_stride_t=1024,
                q_out_stride_h=128, k_out=A, k_out_stride_t=256, k_out_stride_h=128, d_status=None, stream=None)
    assert set(over) <= set(args)
    return {**args, **over}


@no_gpu_only
@pytest.mark.parametrize("over,needle", [
    (dict(num_tokens=-1), "num_tokens < 0"),
    (dict(num_heads=0), "must be positive"),
    (dict(num_kv_heads=0), "must be positive"),
    (dict(head_size=8), "head_size"),
    (dict(head_size=264), "head_size"),
    (dict(head_size=288), "head_size"),
    (dict(rot_dim=8), "rot_dim"),
    (dict(rot_dim=-16), "rot_dim"),
    (dict(rot_dim=144), "rot_dim"),
    (dict(num_tokens=1 << 28), "below 2^31"),
    (dict(q=A + 8), "q must be"),
    (dict(k=None), "k must be"),
    (dict(q_stride_h=64), "q strides"),
    (dict(k_stride_t=-256), "k strides"),
    (dict(q_out=None), "q_out must be"),
    (dict(q_out_stride_t=1016), "rows must not overlap"),
    (dict(k_out_stride_t=0), "rows must not overlap"),
    (dict(q_weight=None), "q_weight / k_weight"),
    (dict(k_weight=A + 4), "q_weight / k_weight"),
    (dict(positions=A + 4), "positions"),
    (dict(max_position=0), "max_position"),
    (dict(cos_sin=None), "cos_sin"),
    (dict(cos_sin=A + 4), "cos_sin"),
    (dict(cos_sin_stride=124), "cos_sin"),
    (dict(cos_sin_stride=130), "cos_sin"),
    (dict(eps=-1e-6), "eps"),
    (dict(eps=float("nan")), "eps"),
    (dict(d_status=A + 2), "d_status"),
])
def test_norm_rope_rejects_bad_arguments_on_host(lib, over, needle):
    rejected(lib, "kvq_qk_norm_rope", norm_args(**over), needle)


def compact_args(**over):
    args = dict(kv_cache=A, num_layers=2, layer_stride=64 * 2 * 2304, num_pages=64, block_size=16, layout=0,
                num_kv_heads=2, head_size=128, query_start=A, seq_lens=A, batch_size=4, accepted=A, accepted_stride=8,
                accepted_lens=A, max_accepted=8, block_table=A, block_table_stride=16, block_table_width=16,
                d_status=None, stream=None)
    assert set(over) <= set(args)
    return {**args, **over}


@no_gpu_only
@pytest.mark.parametrize("over,needle", [
    (dict(num_layers=-1), "must be >= 0"),
    (dict(batch_size=-1), "must be >= 0"),
    (dict(max_accepted=-1), "must be >= 0"),
    (dict(head_size=24), "head_size"),
    (dict(head_size=1040), "head_size"),
    (dict(layout=-1), "layout"),
    (dict(kv_cache=None), "kv_cache"),
    (dict(kv_cache=A + 8), "kv_cache"),
    (dict(num_pages=0), "num_pages"),
    (dict(block_size=0), "block_size"),
    (dict(num_kv_heads=0), "num_kv_heads"),
    (dict(block_size=1, num_kv_heads=1, head_size=16), "multiple of 8"),
    (dict(num_layers=65536, layer_stride=1 << 30), "65535 layers"),
    (dict(num_kv_heads=32768), "32767 heads"),
    (dict(layer_stride=64 * 2 * 2304 - 16), "layer_stride"),
    (dict(layer_stride=64 * 2 * 2304 + 8), "layer_stride"),
    (dict(batch_size=65536), "at most 65535"),
    (dict(query_start=None), "non-NULL"),
    (dict(block_table_width=0), "block_table_width"),
    (dict(block_table_stride=15), "block_table_stride"),
    (dict(accepted=None), "accepted"),
    (dict(accepted_lens=A + 2), "accepted"),
    (dict(accepted_stride=7), "accepted_stride"),
    (dict(d_status=A + 2), "d_status"),
])
def test_compaction_rejects_bad_arguments_on_host(lib, over, needle):
    rejected(lib, "kvq_compact_drafts_nvfp4_per_head", compact_args(**over), needle)


@no_gpu_only
def test_empty_norm_and_compaction_do_nothing(lib):
    assert lib.kvq_qk_norm_rope(*norm_args(num_tokens=0, q=None, k=None).values()) == 0
    for over in (dict(num_layers=0), dict(batch_size=0), dict(max_accepted=0)):
        assert lib.kvq_compact_drafts_nvfp4_per_head(*compact_args(kv_cache=None, **over).values()) == 0


# --------------------------------------------------------------------------
# the Python calls
# --------------------------------------------------------------------------

def test_python_calls_refuse_cpu_tensors_and_other_objects(kvq):
    """CPU tensors never reach a kernel: each call names the argument."""
    bf, i32 = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(4, 2, 16, 2, 72, dtype=torch.uint8)
    one = torch.ones(1)
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        kvq.kvq_window_attention_nvfp4_per_head(bf, i32, i32, i32, cache, one, one, 1.0, 1, 1)
    with pytest.raises(ValueError, match="q: expected a tensor"):
        kvq.kvq_window_attention_nvfp4_per_head(np.zeros((2, 4, 128)), i32, i32, i32, cache, one, one, 1.0, 1, 1)
    with pytest.raises(ValueError, match="tree_mask: expected a tensor"):
        kvq.kvq_tree_attention_nvfp4_per_head(bf, i32, i32, None, i32, cache, one, one, 1.0, 1, 1)
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        kvq.kvq_tree_attention_nvfp4_per_head(bf, i32, i32, i32, i32, cache, one, one, 1.0, 1, 1)
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        kvq.kvq_qk_norm_rope(bf, bf, bf, bf, i32, one, 1e-6)
    with pytest.raises(ValueError, match="kv_cache: expected a CUDA tensor"):
        kvq.kvq_compact_drafts_nvfp4_per_head(cache, i32, i32, i32, i32, i32)
    with pytest.raises(TypeError):
        kvq.kvq_qk_norm_rope(bf)


def test_binding_refuses_a_library_without_the_entry_points(kvq):
    native = kvq._load_native()
    with pytest.raises(KeyError):
        native.bind({})
    with pytest.raises(TypeError, match="wrong number of arguments"):
        native.attention(None)


# --------------------------------------------------------------------------
# the plain reference
# --------------------------------------------------------------------------

def test_reference_e4m3_is_torch_e4m3():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.e4m3(codes), want)


def test_reference_bf16_is_torch_bf16():
    x = np.concatenate([np.float32([0, 1, -1, 1.00390625, 1.01171875, 3.4e38]),
                        np.random.default_rng(0).standard_normal(1000, dtype=np.float32)])
    t = torch.from_numpy(x).bfloat16()
    np.testing.assert_array_equal(ref.to_bf16(x).view(np.int16), t.view(torch.int16).numpy())
    np.testing.assert_array_equal(ref.bf16(ref.to_bf16(x)), t.double().numpy())


def test_reference_attention_by_hand():
    """Two keys, one hidden: the visible one's value and score come out."""
    rng = np.random.default_rng(1)
    cache = ref.Cache(1, 2, 2, 1, 64, "NHD", rng)
    q = rng.standard_normal((1, 1, 64))
    out, lse, _, _ = ref.attention(cache, q, [0, 1], [2], np.array([[1]]), 0.5, 2.0, 0.25, window=1)
    k, v = cache.entry(1, 0, 1, 0), cache.entry(1, 1, 1, 0)
    np.testing.assert_allclose(out[0, 0], 2.0 * v, rtol=1e-12)
    np.testing.assert_allclose(lse[0, 0], 0.125 * (q[0, 0] @ k), rtol=1e-12)
