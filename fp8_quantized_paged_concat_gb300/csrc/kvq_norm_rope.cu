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
// them.  A pair's other half, when it is rot/2 away, sits rot/16 lanes on:
// its raw bf16 values come by four shuffles and are normalised again with
// that lane's weights, which halves the shuffled words against exchanging
// normalised fp32 values.  A lane group works on kHeads heads of one token,
// whose loads are all issued before the first is used; the table's row and
// the weights are loaded once for them.
#include "kvq_device.cuh"
#include "kvq_launch.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;

struct Values {
  float v[8];
};

__device__ __forceinline__ Values unpack8(const uint4& w) {
  return {{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w),
           bf16_hi(w.w)}};
}

// kLanes: lanes of a head; kHeads: heads of one token per lane group.
template <int kLanes, int kHeads, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormRopeArgs a, FastDiv chunk_div) {
  const uint32_t group = static_cast<uint32_t>((static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes);
  const int li = threadIdx.x % kLanes;
  // group -> (token, chunk of kHeads heads); the query heads, then the key heads
  const uint32_t token = chunk_div.div(group);
  const int head0 = static_cast<int>(group - token * chunk_div.d) * kHeads;
  const int total = a.num_heads + a.num_kv_heads;
  const bool live_token = token < a.num_tokens;
  const bool live_lane = live_token && 8 * li < a.head_size;

  uint4 raw[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = head0 + j;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (live_lane && h < total) {
      const __nv_bfloat16* x =
          h < a.num_heads
              ? static_cast<const __nv_bfloat16*>(a.q) + token * a.q_stride_t + h * a.q_stride_h
              : static_cast<const __nv_bfloat16*>(a.k) + token * a.k_stride_t + (h - a.num_heads) * a.k_stride_h;
      raw[j] = ld_stream16(x + 8 * li);
    }
  }

  const int64_t pos = live_token ? __ldg(a.positions + token) : 0;
  const bool bad = live_token && (pos < 0 || pos >= a.max_position);
  if (bad && li == 0 && head0 == 0) report(a.status, KVQ_STATUS_BAD_INDEX);
  const bool live = live_lane && !bad;

  // the lane's cosines and sines: of its 8 dimensions' pairs (the 4 pairs it
  // holds, each twice, when interleaved)
  const int half = a.rot_dim / 2;
  const bool rotated = 8 * li < a.rot_dim;
  const bool second = !kInterleaved && 8 * li >= half;
  Values co{}, si{};
  if (live && rotated) {
    const float* row = a.cos_sin + pos * a.cos_sin_stride;
    if constexpr (kInterleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * li));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + 4 * li));
      co = {{c.x, c.x, c.y, c.y, c.z, c.z, c.w, c.w}};
      si = {{s.x, s.x, s.y, s.y, s.z, s.z, s.w, s.w}};
    } else {
      const float4* c = reinterpret_cast<const float4*>(row + 8 * li - (second ? half : 0));
      const float4* s = reinterpret_cast<const float4*>(row + half + 8 * li - (second ? half : 0));
      const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
      co = {{c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w}};
      si = {{s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w}};
    }
  }
  // a pair's other half: rot/16 lanes on (first half) or back (second half)
  const int partner = kInterleaved || !rotated ? li : second ? li - half / 8 : li + half / 8;

  uint4 wq[2] = {}, wk[2] = {};                // own and partner's weights, per side
  if (live_lane) {
    const uint4* q = static_cast<const uint4*>(a.q_weight);
    const uint4* k = static_cast<const uint4*>(a.k_weight);
    if (head0 < a.num_heads) {
      wq[0] = __ldg(q + li);
      if constexpr (!kInterleaved) wq[1] = __ldg(q + partner);
    }
    if (head0 + kHeads > a.num_heads) {
      wk[0] = __ldg(k + li);
      if constexpr (!kInterleaved) wk[1] = __ldg(k + partner);
    }
  }

  const float inv_dim = 1.0f / static_cast<float>(a.head_size);
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = head0 + j;
    const bool is_q = h < a.num_heads;
    Values x = unpack8(raw[j]);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __fmaf_rn(x.v[i], x.v[i], ss);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o, kLanes);
    const float r = rsqrtf(__fmaf_rn(ss, inv_dim, a.eps));
    const Values w = unpack8(is_q ? wq[0] : wk[0]);
    Values y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y.v[i] = x.v[i] * r * w.v[i];
    Values z = y;
    if constexpr (kInterleaved) {
      if (rotated) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          z.v[i] = y.v[i] * co.v[i] - y.v[i + 1] * si.v[i];
          z.v[i + 1] = y.v[i + 1] * co.v[i] + y.v[i] * si.v[i];
        }
      }
    } else {
      uint4 other;
      other.x = __shfl_sync(kFull, raw[j].x, partner, kLanes);
      other.y = __shfl_sync(kFull, raw[j].y, partner, kLanes);
      other.z = __shfl_sync(kFull, raw[j].z, partner, kLanes);
      other.w = __shfl_sync(kFull, raw[j].w, partner, kLanes);
      if (rotated) {
        const Values p = unpack8(other), wp = unpack8(is_q ? wq[1] : wk[1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float yp = p.v[i] * r * wp.v[i];
          z.v[i] = y.v[i] * co.v[i] + (second ? yp : -yp) * si.v[i];
        }
      }
    }
    if (live && h < total) {
      __nv_bfloat16* o =
          is_q ? static_cast<__nv_bfloat16*>(a.q_out) + token * a.q_out_stride_t + h * a.q_out_stride_h
               : static_cast<__nv_bfloat16*>(a.k_out) + token * a.k_out_stride_t + (h - a.num_heads) * a.k_out_stride_h;
      st16(o + 8 * li, make_uint4(pack_bf16x2(z.v[0], z.v[1]), pack_bf16x2(z.v[2], z.v[3]),
                                  pack_bf16x2(z.v[4], z.v[5]), pack_bf16x2(z.v[6], z.v[7])));
    }
  }
}

template <int kLanes, int kHeads>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t stream) {
  const int chunks = (a.num_heads + a.num_kv_heads + kHeads - 1) / kHeads;
  const uint64_t threads = static_cast<uint64_t>(a.num_tokens) * chunks * kLanes;
  const unsigned blocks = static_cast<unsigned>((threads + kThreads - 1) / kThreads);
  const FastDiv div = FastDiv::make(static_cast<uint32_t>(chunks));
  if (a.interleaved)
    qk_norm_rope_kernel<kLanes, kHeads, true><<<blocks, kThreads, 0, stream>>>(a, div);
  else
    qk_norm_rope_kernel<kLanes, kHeads, false><<<blocks, kThreads, 0, stream>>>(a, div);
  return cudaGetLastError();
}

template <int kLanes>
cudaError_t launch_heads(const NormRopeArgs& a, int num_sms, cudaStream_t stream) {
  // Four heads per lane group share one table row and keep four loads in
  // flight; a call too small to fill the GPU that way takes one head each.
  const int64_t threads = a.num_tokens * ((a.num_heads + a.num_kv_heads + 3) / 4) * kLanes;
  return threads >= static_cast<int64_t>(num_sms) * 1024 ? launch<kLanes, 4>(a, stream) : launch<kLanes, 1>(a, stream);
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
