// kvq_append.cu -- the new tokens of every request: queries and keys rotated
// by their positions, keys and values quantized to e4m3 and appended to the
// paged per-head cache, whose pages have one power-of-two scale per side and
// head.
//
// For a pair (a, b) of a head with its token's cosine c and sine s:
//   (a, b) -> (a c - b s, b c + a s), every product and sum one fp32 rounding,
// with pair j = (j, j + rot/2), or (2j, 2j + 1) when interleaved.  For a page,
// side and head whose new values y have the largest magnitude A:
//   e = the least integer with A <= 448 * 2^e, in [-60, 60];
//   with entries before the first new one in the page: e = max(e, the page's
//   own), and where that grows, those entries' codes become e4m3(value *
//   2^(old - e)), exact but for e4m3's subnormals;
//   code = e4m3(y * 2^-e), scale byte = e + 127.
// A power of two costs nothing: e4m3 has the same relative precision at every
// magnitude, and the scale only has to keep the largest value in range.
//
// Bound: HBM (keys and values read once and written as one byte each, queries
// read and written).  One warp, or four or eight, per (page, side, head), as
// many as keep the page's new tokens in registers between the largest magnitude
// and the codes (a page of more is read twice).  D / 8 lanes hold a token's
// head, 8 values (16 bytes) each, eight tokens a lane, whose loads are all
// under way at once; a pair's other half, rot/16 lanes on, comes by shuffles of
// the raw bf16 values.  The queries are other CTAs' work in the same launch: up
// to 8 heads of a token per lane group, which share the token's row of the
// table.  Measured (32 query heads, 8 key heads of 128): 4 x 4096 tokens, 411
// MB, into pages of 32 70 us = 5.9 TB/s, of 64 75 us = 5.5; 128 decoded tokens
// 3.3 us and one 2.4 in a graph, of which the launch and three dependent loads
// (the request, its page, the scale) are most.
#include <algorithm>

#include "kvq_dependent.cuh"
#include "kvq_device.cuh"
#include "kvq_launch.h"

namespace kvq {
namespace {

constexpr int kManyHeads = 8;                // query heads per lane group of a call that fills the GPU

__host__ __device__ constexpr int threads_of(int warps) { return warps == 8 ? 256 : 128; }

// 8 values as fp32 pairs.
struct Values {
  float2 v[4];
};

__device__ __forceinline__ Values unpack8(const uint4& w) {
  return {{make_float2(bf16_lo(w.x), bf16_hi(w.x)), make_float2(bf16_lo(w.y), bf16_hi(w.y)),
           make_float2(bf16_lo(w.z), bf16_hi(w.z)), make_float2(bf16_lo(w.w), bf16_hi(w.w))}};
}

__device__ __forceinline__ uint4 pack8(const Values& y) {
  return make_uint4(pack_bf16x2(y.v[0].x, y.v[0].y), pack_bf16x2(y.v[1].x, y.v[1].y),
                    pack_bf16x2(y.v[2].x, y.v[2].y), pack_bf16x2(y.v[3].x, y.v[3].y));
}

// One token's rotation as a lane needs it: its value d becomes x_d own_d +
// x'_d other_d, x'_d the other half of d's pair.
struct Turn {
  Values own, other;
};

// Lane li of a head: where its pairs' other halves are.
template <bool kInterleaved>
struct Place {
  int partner;
  bool rotated, second;
  __device__ __forceinline__ Place(int li, int rot_dim) {
    rotated = 8 * li < rot_dim;
    second = !kInterleaved && 8 * li >= rot_dim / 2;
    partner = kInterleaved || !rotated ? li : second ? li - rot_dim / 16 : li + rot_dim / 16;
  }
};

template <bool kInterleaved>
__device__ __forceinline__ Turn load_turn(const AppendArgs& a, const Place<kInterleaved>& at, int li, int64_t pos) {
  Turn t;
  const int half = a.rot_dim / 2;
  const float* row = a.cos_sin + pos * a.cos_sin_stride;
  if constexpr (kInterleaved) {
    const float4 c = load_global(reinterpret_cast<const float4*>(row + 4 * li));
    const float4 s = load_global(reinterpret_cast<const float4*>(row + half + 4 * li));
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.own.v[i] = make_float2(cs[i], cs[i]);
      t.other.v[i] = make_float2(-sn[i], sn[i]);
    }
  } else {
    const float4* c = reinterpret_cast<const float4*>(row + 8 * li - (at.second ? half : 0));
    const float4* s = reinterpret_cast<const float4*>(row + half + 8 * li - (at.second ? half : 0));
    const float sign = at.second ? 1.0f : -1.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c4 = load_global(c + i), s4 = load_global(s + i);
      t.own.v[2 * i] = make_float2(c4.x, c4.y);
      t.own.v[2 * i + 1] = make_float2(c4.z, c4.w);
      t.other.v[2 * i] = make_float2(sign * s4.x, sign * s4.y);
      t.other.v[2 * i + 1] = make_float2(sign * s4.z, sign * s4.w);
    }
  }
  return t;
}

// A lane's eight values of a head, rotated.  Every lane of the warp comes here.
template <int kLanes, bool kInterleaved>
__device__ __forceinline__ Values rotate(const uint4& raw, const Place<kInterleaved>& at, const Turn& t) {
  const Values x = unpack8(raw);
  Values p;
  if constexpr (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p.v[i] = make_float2(x.v[i].y, x.v[i].x);
  } else {
    uint4 w;
    w.x = __shfl_sync(kFull, raw.x, at.partner, kLanes);
    w.y = __shfl_sync(kFull, raw.y, at.partner, kLanes);
    w.z = __shfl_sync(kFull, raw.z, at.partner, kLanes);
    w.w = __shfl_sync(kFull, raw.w, at.partner, kLanes);
    p = unpack8(w);
  }
  if (!at.rotated) return x;
  Values y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (not as packed pairs, whose product and sum the compiler was seen to fuse)
    y.v[i].x = __fadd_rn(__fmul_rn(x.v[i].x, t.own.v[i].x), __fmul_rn(p.v[i].x, t.other.v[i].x));
    y.v[i].y = __fadd_rn(__fmul_rn(x.v[i].y, t.own.v[i].y), __fmul_rn(p.v[i].y, t.other.v[i].y));
  }
  return y;
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The least e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), in [-60, 60].
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u);
  return max(KVQ_FP8_SCALE_MIN_EXP, min(KVQ_FP8_SCALE_MAX_EXP, e));
}
__device__ __forceinline__ int stored_exponent(uint32_t byte) {
  return max(KVQ_FP8_SCALE_MIN_EXP, min(KVQ_FP8_SCALE_MAX_EXP, static_cast<int>(byte) - KVQ_FP8_SCALE_BIAS));
}

__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b, float f) {
  const float2 s = make_float2(f, f);
  const float2 x = fmul2(a, s), y = fmul2(b, s);
  return cvt_e4m3x2(x.x, x.y) | cvt_e4m3x2(y.x, y.y) << 16;
}

// The codes of a word, each value times f.
__device__ __forceinline__ uint32_t recode(uint32_t w, float f) {
  const float2 lo = __half22float2(e4m3x2_to_half2(w & 0xFFFFu)), hi = __half22float2(e4m3x2_to_half2(w >> 16));
  return e4m3x4(lo, hi, f);
}

// kWarps warps (of number `warp`, all of a CTA, or one): the new entries of one
// page, side and head; a lane keeps kHeld tokens' between the two looks at them.
template <int kLanes, int kWarps, int kHeld, bool kInterleaved>
__device__ __forceinline__ void append_page(const AppendArgs& a, int b, int64_t token0, int32_t n, int32_t len,
                                            uint32_t unit, int warp, int lane) {
  constexpr int kTokens = 32 / kLanes;               // of a warp at a time
  constexpr int kAtOnce = kTokens * kWarps, kChunk = kAtOnce * kHeld;
  constexpr int D = 8 * kLanes;
  const uint32_t side_heads = 2u * a.num_kv_heads;
  const uint32_t ordinal = unit / side_heads, sh = unit - ordinal * side_heads;
  const bool is_v = sh >= static_cast<uint32_t>(a.num_kv_heads);
  const uint32_t head = sh - (is_v ? a.num_kv_heads : 0);
  const int32_t first = len - n;                     // position of the first new token
  const uint32_t col = a.block_div.div(static_cast<uint32_t>(first)) + ordinal;
  const int64_t base = static_cast<int64_t>(col) * a.block_size;
  if (base >= len) return;                           // past the request's last page
  // Its new entries are [held, end).  (Entries are counted within their page:
  // steps past the last one would wrap as positions of a sequence near 2^31.)
  const int32_t held = static_cast<int32_t>(max(int64_t{0}, first - base));
  const int32_t end = static_cast<int32_t>(min(static_cast<int64_t>(a.block_size), len - base));
  const int64_t page_token = token0 + (base - first);          // the token of entry 0, were it new
  int32_t id = -1;
  if (col < static_cast<uint32_t>(a.block_table_width)) id = load_global(a.block_table + b * a.block_table_stride + col);

  const int li = lane % kLanes, sub = warp * kTokens + lane / kLanes;
  const Place<kInterleaved> at(li, a.rot_dim);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? a.v : a.k) +
                             head * (is_v ? a.v_stride_h : a.k_stride_h) + 8 * li;
  const int64_t stride = is_v ? a.v_stride_t : a.k_stride_t;
  // The lane's values of the entries p + sub, kAtOnce on, ..., every load under
  // way before the first is used; bit j of `live`: there is one, and its rotation
  // position is in the table.
  Values y[kHeld];
  uint32_t live;
  auto values = [&](int32_t p) {
    uint4 raw[kHeld];
    int64_t pos[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int32_t q = p + sub + kAtOnce * j;
      raw[j] = make_uint4(0, 0, 0, 0);
      pos[j] = -1;
      if (q < end) {
        const int64_t token = page_token + q;
        raw[j] = load_global(reinterpret_cast<const uint4*>(src + token * stride));
        pos[j] = load_global(a.positions + token);
      }
    }
    live = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const bool ok = pos[j] >= 0 && pos[j] < a.max_position;
      if (!ok && li == 0 && p + sub + kAtOnce * j < end) report(a.status, KVQ_STATUS_BAD_INDEX);
      live |= ok ? 1u << j : 0u;
      if (is_v) {
        y[j] = unpack8(raw[j]);
      } else {
        Turn t{};
        if (ok && at.rotated) t = load_turn<kInterleaved>(a, at, li, pos[j]);
        y[j] = rotate<kLanes, kInterleaved>(raw[j], at, t);
      }
    }
  };

  float amax = 0.0f;
  for (int32_t p = held; p < end; p += kChunk) {
    values(p);
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if ((live >> j) & 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(y[j].v[i].x), fabsf(y[j].v[i].y)));
      }
  }
  const bool there = id >= 0 && id < a.num_pages;
  if (!there && warp == 0 && lane == 0) report(a.status, KVQ_STATUS_BAD_INDEX);
  uint8_t* scale = a.scales + (static_cast<int64_t>(there ? id : 0) * side_heads + sh);
  uint8_t* region = a.cache + (2 * static_cast<uint64_t>(there ? id : 0) + is_v) * a.region;
  const int old = there && held > 0 ? stored_exponent(load_global(scale)) : KVQ_FP8_SCALE_MIN_EXP;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  if constexpr (kWarps > 1) {
    __shared__ float most[kWarps];
    if (lane == 0) most[warp] = amax;
    __syncthreads();                                 // (and every warp has read the scale)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, most[w]);
  }
  __syncwarp();
  const int e = max(scale_exponent(amax), old);
  if (there) {
    if (held > 0 && e > old) {
      const float f = power_of_two(old - e);
      constexpr int kChunks = D / 16;
      for (int i = warp * 32 + lane; i < held * kChunks; i += 32 * kWarps) {
        const uint32_t row = static_cast<uint32_t>(i / kChunks) * a.row_offset + head * a.row_head;
        uint4* w = reinterpret_cast<uint4*>(region + static_cast<uint64_t>(row) * D) + i % kChunks;
        const uint4 x = *w;
        *w = make_uint4(recode(x.x, f), recode(x.y, f), recode(x.z, f), recode(x.w, f));
      }
    }
    if (warp == 0 && lane == 0) *scale = static_cast<uint8_t>(e + KVQ_FP8_SCALE_BIAS);
  }
  const bool keep = !is_v && a.k_out != nullptr;
  if (!there && !keep) return;
  const float f = power_of_two(-e);
  const bool again = end - held > kChunk;              // more tokens than are held
  for (int32_t p = held; p < end; p += kChunk) {
    if (again) values(p);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (!((live >> j) & 1)) continue;
      const int32_t q = p + sub + kAtOnce * j;
      if (there) {
        const uint32_t row = static_cast<uint32_t>(q) * a.row_offset + head * a.row_head;
        st8(region + static_cast<uint64_t>(row) * D + 8 * li,
            make_uint2(e4m3x4(y[j].v[0], y[j].v[1], f), e4m3x4(y[j].v[2], y[j].v[3], f)));
      }
      if (keep)
        st16(static_cast<__nv_bfloat16*>(a.k_out) + (page_token + q) * a.k_out_stride_t + head * a.k_out_stride_h +
                 8 * li, pack8(y[j]));
    }
  }
}

// One lane group: up to kHeads query heads of one token.
template <int kLanes, int kHeads, bool kInterleaved>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, int64_t token0, int32_t n, uint64_t thread) {
  const uint32_t group = static_cast<uint32_t>(thread / kLanes);
  const int li = static_cast<int>(thread % kLanes);
  const uint32_t chunks = (a.num_heads + kHeads - 1) / kHeads;
  const uint32_t i = group / chunks, head0 = (group - i * chunks) * kHeads;
  const int heads = min(kHeads, static_cast<int>(a.num_heads - head0));
  const bool in = i < static_cast<uint32_t>(n);
  const int64_t token = token0 + i;
  const __nv_bfloat16* src =
      static_cast<const __nv_bfloat16*>(a.q) + token * a.q_stride_t + head0 * a.q_stride_h + 8 * li;
  uint4 raw[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
    raw[j] = in && j < heads ? load_global(reinterpret_cast<const uint4*>(src + j * a.q_stride_h)) : make_uint4(0, 0, 0, 0);
  const int64_t pos = in ? load_global(a.positions + token) : 0;
  const bool live = in && pos >= 0 && pos < a.max_position;
  if (in && !live && li == 0) report(a.status, KVQ_STATUS_BAD_INDEX);
  const Place<kInterleaved> at(li, a.rot_dim);
  Turn t{};
  if (live && at.rotated) t = load_turn<kInterleaved>(a, at, li, pos);
  __nv_bfloat16* dst =
      static_cast<__nv_bfloat16*>(a.q_out) + token * a.q_out_stride_t + head0 * a.q_out_stride_h + 8 * li;
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const Values y = rotate<kLanes, kInterleaved>(raw[j], at, t);
    if (live && j < heads) st16(dst + j * a.q_out_stride_h, pack8(y));
  }
}

// kWarps: warps of a page, side and head.
template <int kLanes, int kWarps, int kHeld, int kHeads, bool kInterleaved>
__global__ void __launch_bounds__(threads_of(kWarps), kWarps == 8 ? 3 : kWarps == 4 && kHeld == 2 ? 8 : 6)
    append_kernel(const AppendArgs a, uint32_t page_ctas, uint32_t units) {
  wait_for_previous();
  allow_dependents();
  constexpr int kThreads = threads_of(kWarps);
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t q0 = load_global(a.query_start + b), q1 = load_global(a.query_start + b + 1);
  const int32_t len = max(0, load_global(a.seq_lens + b));
  const int64_t n = static_cast<int64_t>(q1) - q0;
  if (q0 < 0 || n < 0 || q1 > a.num_tokens || n > a.max_query_len || n > len) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, KVQ_STATUS_BAD_BATCH);
    return;
  }
  if (n == 0) return;
  if (blockIdx.x < page_ctas) {
    const uint32_t unit = kWarps == 1 ? blockIdx.x * (kThreads / 32) + warp : blockIdx.x;
    if (unit < units)
      append_page<kLanes, kWarps, kHeld, kInterleaved>(a, b, q0, static_cast<int32_t>(n), len, unit, kWarps == 1 ? 0 : warp, lane);
  } else {
    rotate_queries<kLanes, kHeads, kInterleaved>(a, q0, static_cast<int32_t>(n),
                                                 static_cast<uint64_t>(blockIdx.x - page_ctas) * kThreads + threadIdx.x);
  }
}

template <int kLanes, int kWarps, int kHeld, int kHeads>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  constexpr int kThreads = threads_of(kWarps), kUnits = kThreads / (32 * kWarps);
  const int64_t pages = (static_cast<int64_t>(a.max_query_len) + a.block_size - 2) / a.block_size + 1;
  const int64_t units = pages * 2 * a.num_kv_heads, page_ctas = (units + kUnits - 1) / kUnits;
  const int64_t chunks = (a.num_heads + kHeads - 1) / kHeads;
  const int64_t query_ctas =
      a.q == nullptr ? 0 : (static_cast<int64_t>(a.max_query_len) * chunks * kLanes + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(page_ctas + query_ctas), static_cast<unsigned>(a.batch_size));
  return launch_dependent(
      a.interleaved ? append_kernel<kLanes, kWarps, kHeld, kHeads, true>
                    : append_kernel<kLanes, kWarps, kHeld, kHeads, false>,
      grid, kThreads, 0, 1, stream, a, static_cast<uint32_t>(page_ctas), static_cast<uint32_t>(units));
}

template <int kLanes>
cudaError_t launch_size(const AppendArgs& a, int num_sms, cudaStream_t stream) {
  // As many warps as hold a page's new tokens between the two looks at them, and
  // no more (us at D = 128, 8 key heads, 32 query heads; 1 warp x 1 token a lane,
  // 1 x 4, 4 x 2, 4 x 4, 8 x 4): 128 requests x 1 token 3.3, 4.9, -, 8.4, 14; 128 x
  // 4 tokens 5.5, 5.7, 8.9, 11, 19; pages of 16: 32 x 16 tokens 9.1, 9.4, 5.8, 6.3,
  // 9.0, 4 x 4096 82, 80, 78, 87, 140; pages of 32: 32 x 32 17, 16, -, 8.4, 10, 4 x
  // 4096 95, 83, 78, 70, 96; pages of 64: 16 x 64 33, 27, 11, 10, 8.0, 16 x 500 70,
  // 60, 41, 40, 38, 4 x 4096 116, 101, 74, 73, 75.
  const int64_t tokens = std::min<int64_t>(a.max_query_len, a.block_size);
  constexpr int kAtOnce = 32 / kLanes;
  // Query heads of a lane group: eight where the call has the lanes for it (256
  // tokens x 32 heads 4.8 us, one head each 5.2; 180 tokens 4.0 / 4.3; 128 tokens
  // 3.9 / 3.3; 4 x 4096 70 / 119).
  const int64_t chunks = (a.num_heads + kManyHeads - 1) / kManyHeads;
  const bool many = a.num_tokens * chunks * kLanes >= static_cast<int64_t>(num_sms) * 64;
  if (tokens <= kAtOnce) return many ? launch<kLanes, 1, 1, kManyHeads>(a, stream) : launch<kLanes, 1, 1, 1>(a, stream);
  if (tokens <= 4 * kAtOnce) return many ? launch<kLanes, 1, 4, kManyHeads>(a, stream) : launch<kLanes, 1, 4, 1>(a, stream);
  if (tokens <= 8 * kAtOnce) return many ? launch<kLanes, 4, 2, kManyHeads>(a, stream) : launch<kLanes, 4, 2, 1>(a, stream);
  if (tokens <= 16 * kAtOnce) return many ? launch<kLanes, 4, 4, kManyHeads>(a, stream) : launch<kLanes, 4, 4, 1>(a, stream);
  return launch<kLanes, 8, 4, kManyHeads>(a, stream);
}

}  // namespace

cudaError_t launch_rope_append(const AppendArgs& a, int num_sms, cudaStream_t stream) {
  switch (a.head_size) {
    case 64: return launch_size<8>(a, num_sms, stream);
    case 128: return launch_size<16>(a, num_sms, stream);
    default: return launch_size<32>(a, num_sms, stream);
  }
}

}  // namespace kvq
