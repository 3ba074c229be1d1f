// kvq_norm_rope.cu -- RMS norm of every query and key head and the rotation
// by its token's position, in one pass over the values.
//
// For a head x of D values, its side's weight w and the token's position p:
//   y_d = x_d * w_d / sqrt(sum_i x_i^2 / D + eps)
//   (a, b) -> (a cos - b sin, b cos + a sin)    for the rotated pairs of y
// with pair j = (j, j + rot/2), or (2j, 2j + 1) when interleaved, and row p
// of the caller's table (cosines of the rot/2 pairs, then their sines);
// dimensions from rot on are only normalised.  All of it in fp32, one bf16
// rounding at the end.
//
// Bound: HBM (each value is read and written once, 4 bytes in all; about 6
// operations).  A head takes L = D / 8 lanes rounded up to a power of two, 8
// values (16 bytes) each; the sum of squares is a shuffle reduction over
// them.  A lane group works on up to 8 heads of one side of one token, whose
// loads are all issued before the first is used.  Weights, cosines, sines and
// signs are folded once per group into two factors per dimension, so that a
// value costs two multiplications and one fused multiply-add.  A pair's other
// half, when it is rot/2 away, sits rot/16 lanes on: its raw bf16 values come
// by four shuffles.  16384 tokens x (32 + 8) heads of 128: 57 us, 6.1 TB/s
// (normalised fp32 values with unfused factors: 74 us).
#include "kvq_dependent.cuh"
#include "kvq_device.cuh"
#include "kvq_launch.h"

namespace kvq {
namespace {

constexpr int kThreads = 128;
constexpr int kManyHeads = 8;                // heads per lane group of a call that fills the GPU

// 8 bf16 values as fp32 pairs.
struct Values {
  float2 v[4];
};

__device__ __forceinline__ Values unpack8(const uint4& w) {
  return {{make_float2(bf16_lo(w.x), bf16_hi(w.x)), make_float2(bf16_lo(w.y), bf16_hi(w.y)),
           make_float2(bf16_lo(w.z), bf16_hi(w.z)), make_float2(bf16_lo(w.w), bf16_hi(w.w))}};
}

// kLanes: lanes of a head; kHeads: heads of one token per lane group.
template <int kLanes, int kHeads, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 6) qk_norm_rope_kernel(const NormRopeArgs a, FastDiv chunk_div,
                                                                   int q_chunks) {
  wait_for_previous();
  allow_dependents();
  const uint32_t group = static_cast<uint32_t>((static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes);
  const int li = threadIdx.x % kLanes;
  // group -> (token, chunk of kHeads heads): the query side's chunks, then the key side's
  const uint32_t token = chunk_div.div(group);
  const int chunk = static_cast<int>(group - token * chunk_div.d);
  const bool is_q = chunk < q_chunks;
  const int head0 = (is_q ? chunk : chunk - q_chunks) * kHeads;
  const int heads = min(kHeads, (is_q ? a.num_heads : a.num_kv_heads) - head0);
  const bool live_token = token < a.num_tokens;
  const bool live_lane = live_token && 8 * li < a.head_size;
  const int64_t in_h = is_q ? a.q_stride_h : a.k_stride_h;
  const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(is_q ? a.q : a.k) +
                            token * (is_q ? a.q_stride_t : a.k_stride_t) + head0 * in_h + 8 * li;

  uint4 raw[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
    raw[j] = live_lane && j < heads ? *reinterpret_cast<const uint4*>(in + j * in_h) : make_uint4(0, 0, 0, 0);

  const int64_t pos = live_token ? load_global(a.positions + token) : 0;
  const bool bad = live_token && (pos < 0 || pos >= a.max_position);
  if (bad && li == 0 && chunk == 0) report(a.status, KVQ_STATUS_BAD_INDEX);
  const bool live = live_lane && !bad;

  // A lane's value d becomes r (x_d own_d + x'_d other_d) with r the head's
  // inverse norm, x'_d the other half of d's pair, own = w cos and other = the
  // other half's w times -sin (first half) or sin (second half); outside the
  // rotation own = w, other = 0.
  const int half = a.rot_dim / 2;
  const bool rotated = 8 * li < a.rot_dim;
  const bool second = !kInterleaved && 8 * li >= half;
  const int partner = kInterleaved || !rotated ? li : second ? li - half / 8 : li + half / 8;
  Values own{}, other{};
  if (live) {
    const uint4* w = static_cast<const uint4*>(is_q ? a.q_weight : a.k_weight);
    own = unpack8(load_global(w + li));
    if (rotated) {
      const float* row = a.cos_sin + pos * a.cos_sin_stride;
      if constexpr (kInterleaved) {
        const float4 c = load_global(reinterpret_cast<const float4*>(row + 4 * li));
        const float4 s = load_global(reinterpret_cast<const float4*>(row + half + 4 * li));
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          other.v[i] = make_float2(-own.v[i].y * sn[i], own.v[i].x * sn[i]);
          own.v[i] = fmul2(own.v[i], make_float2(cs[i], cs[i]));
        }
      } else {
        other = unpack8(load_global(w + partner));
        const float2* c = reinterpret_cast<const float2*>(row + 8 * li - (second ? half : 0));
        const float2* s = reinterpret_cast<const float2*>(row + half + 8 * li - (second ? half : 0));
        const float sign = second ? 1.0f : -1.0f;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float4 c4 = load_global(reinterpret_cast<const float4*>(c + i)), s4 = load_global(reinterpret_cast<const float4*>(s + i));
          own.v[i] = fmul2(own.v[i], make_float2(c4.x, c4.y));
          own.v[i + 1] = fmul2(own.v[i + 1], make_float2(c4.z, c4.w));
          other.v[i] = fmul2(other.v[i], make_float2(sign * s4.x, sign * s4.y));
          other.v[i + 1] = fmul2(other.v[i + 1], make_float2(sign * s4.z, sign * s4.w));
        }
      }
    }
  }
  const int64_t out_h = is_q ? a.q_out_stride_h : a.k_out_stride_h;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_q ? a.q_out : a.k_out) +
                       token * (is_q ? a.q_out_stride_t : a.k_out_stride_t) + head0 * out_h + 8 * li;

  const float inv_dim = 1.0f / static_cast<float>(a.head_size);
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const Values x = unpack8(raw[j]);
    float2 ss2 = fmul2(x.v[0], x.v[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) ss2 = ffma2(x.v[i], x.v[i], ss2);
    float ss = ss2.x + ss2.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o, kLanes);
    const float r = rsqrtf(__fmaf_rn(ss, inv_dim, a.eps));
    Values p;
    if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p.v[i] = make_float2(x.v[i].y, x.v[i].x);
    } else {
      uint4 w;
      w.x = __shfl_sync(kFull, raw[j].x, partner, kLanes);
      w.y = __shfl_sync(kFull, raw[j].y, partner, kLanes);
      w.z = __shfl_sync(kFull, raw[j].z, partner, kLanes);
      w.w = __shfl_sync(kFull, raw[j].w, partner, kLanes);
      p = unpack8(w);
    }
    uint32_t z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = fmul2(ffma2(p.v[i], other.v[i], fmul2(x.v[i], own.v[i])), make_float2(r, r));
      z[i] = pack_bf16x2(y.x, y.y);
    }
    if (live && j < heads) st16(out + j * out_h, make_uint4(z[0], z[1], z[2], z[3]));
  }
}

template <int kLanes, int kHeads>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t stream) {
  const int q_chunks = (a.num_heads + kHeads - 1) / kHeads;
  const int chunks = q_chunks + (a.num_kv_heads + kHeads - 1) / kHeads;
  const uint64_t threads = static_cast<uint64_t>(a.num_tokens) * chunks * kLanes;
  const unsigned blocks = static_cast<unsigned>((threads + kThreads - 1) / kThreads);
  const FastDiv div = FastDiv::make(static_cast<uint32_t>(chunks));
  return launch_dependent(a.interleaved ? qk_norm_rope_kernel<kLanes, kHeads, true> : qk_norm_rope_kernel<kLanes, kHeads, false>,
                          dim3(blocks), kThreads, 0, 1, stream, a, div, q_chunks);
}

template <int kLanes>
cudaError_t launch_heads(const NormRopeArgs& a, int num_sms, cudaStream_t stream) {
  // Eight heads per lane group share one table row and one set of weights and
  // keep eight loads in flight (head size 128, 32 + 8 heads, in a graph: 16384
  // tokens 54 us, with four heads 61, two 75, one 102); a call that gives the
  // SMs less than one CTA each that way takes one head per group (64 tokens:
  // 1.8 against 2.6 us; 256 tokens 2.7 against 2.9; 1024 tokens 6.9 against 4.9).
  const int64_t chunks = (a.num_heads + kManyHeads - 1) / kManyHeads + (a.num_kv_heads + kManyHeads - 1) / kManyHeads;
  return a.num_tokens * chunks * kLanes >= static_cast<int64_t>(num_sms) * kThreads
             ? launch<kLanes, kManyHeads>(a, stream)
             : launch<kLanes, 1>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int num_sms, cudaStream_t stream) {
  const int lanes = a.head_size / 8;
  if (lanes <= 4) return launch_heads<4>(a, num_sms, stream);
  if (lanes <= 8) return launch_heads<8>(a, num_sms, stream);
  if (lanes <= 16) return launch_heads<16>(a, num_sms, stream);
  return launch_heads<32>(a, num_sms, stream);
}

}  // namespace kvq
