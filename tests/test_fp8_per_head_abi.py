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
