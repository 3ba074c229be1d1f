// kvq_per_head_attention.cuh -- what the two attention kernels over the
// per-head NVFP4 cache share: the requests, the keys a block of query rows
// sees, and the decoding of e2m1 codes.
#pragma once

#include "kvq_dependent.cuh"
#include "kvq_device.cuh"
#include "kvq_launch.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

// The weights of the softmax are kept as 2^(s - m + kShift) in f16, where the
// reference m lags the true maximum by at most kGrow: they stay below 2^14.
constexpr float kGrow = 8.0f;
constexpr float kShift = 6.0f;
constexpr float kMaxWeight = 16384.0f;            // 2^(kShift + kGrow), far below f16's largest value
constexpr float kLn2 = 0.69314718055994530942f;
// Base-2 log-sum-exp of a key range whose CTA gave up: its rows stay unwritten.
constexpr uint32_t kAbandoned = 0x7fc0deadu;

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) { return bits(__hmul2(half2_of(a), half2_of(b))); }
__device__ __forceinline__ uint32_t low_both(uint32_t w) { return bits(__low2half2(half2_of(w))); }
__device__ __forceinline__ uint32_t high_both(uint32_t w) { return bits(__high2half2(half2_of(w))); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) { return bits(__floats2half2_rn(lo, hi)); }

// The four bytes of w (two e2m1 codes each) as f16 pairs: one conversion per
// pair, which takes its byte without a shift.  64 conversions per clock and
// SM, the rate of any integer instruction, so that 8 values cost 4 of them;
// shifts and masks that place the code bits in an f16 cost 11.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// Asynchronous copies into shared memory; `bytes` = kBytes, or 0: zero-filled,
// nothing read.
template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, uint32_t bytes) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" :: "r"(dst), "l"(src), "n"(kBytes), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(kLeft) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

// Scales of values (f16 pairs): a NaN (no write of finite values makes one)
// reads as zero, so that a hidden entry that was never written cannot reach
// any row through a weight of zero.
__device__ __forceinline__ uint32_t finite_scales(uint32_t s) { return s & __heq2_mask(half2_of(s), half2_of(s)); }

// The power of two that brings a query row's largest value to [2^14, 2^15),
// as two factors f[0] f[1], and the one that takes it back, i[0] i[1].
// Rows of zeros, subnormals or infinities stay as they are.
struct RowScale {
  float f[2], i[2];
};
__device__ __forceinline__ RowScale row_scale(float amax) {
  const int ex = static_cast<int>(__float_as_uint(amax) >> 23);
  const int shift = ex == 0 || ex == 255 ? 0 : 127 + 14 - ex;
  const int sh0 = shift / 2, sh1 = shift - sh0;
  return {{__uint_as_float(static_cast<uint32_t>(127 + sh0) << 23), __uint_as_float(static_cast<uint32_t>(127 + sh1) << 23)},
          {__uint_as_float(static_cast<uint32_t>(127 - sh0) << 23), __uint_as_float(static_cast<uint32_t>(127 - sh1) << 23)}};
}

// The keys of one block of query rows: positions [0, sinks) and [lo, hi), in
// steps of kStep.
template <int kStep>
struct Keys {
  int32_t sinks, lo, hi;
  int32_t sink_steps, steps;

  __device__ __forceinline__ int32_t base(int32_t step) const {
    return step * kStep + (step < sink_steps ? 0 : lo - sink_steps * kStep);
  }
  __device__ __forceinline__ int32_t limit(int32_t step) const { return step < sink_steps ? sinks : hi; }
};

// One lane's look-up of a position: its page id, loaded a step before the
// copies that need it start and looked at only there, and its row.
struct LookUp {
  uint32_t row;                // of (position, head) in its page's side region
  int32_t id;                  // page id, -1 where there is none to be had
  bool in;                     // the position is one of the keys
};
__device__ __forceinline__ LookUp look_up_position(const PerHeadAttentionArgs& a, const int32_t* table, uint32_t head_row,
                                                   bool in, uint32_t p) {
  LookUp u;
  const uint32_t col = a.block_div.div(p);
  u.in = in;
  u.row = (p - col * static_cast<uint32_t>(a.block_size)) * static_cast<uint32_t>(a.row_offset) + head_row;
  u.id = -1;
  if (in && col < static_cast<uint32_t>(a.block_table_width)) u.id = load_global(table + col);
  return u;
}
// a + b c in 64 bits, b and c 32 (one instruction).
__device__ __forceinline__ const uint8_t* at_offset(const uint8_t* a, uint32_t b, uint32_t c) {
  return a + static_cast<uint64_t>(b) * c;
}

struct Request {
  int64_t token0;              // its first query token
  int32_t tokens;              // its query tokens
  int64_t first_pos;           // position of its first query token (may be negative)
  bool cut;                    // the sequence goes past the block table
  int32_t len;                 // its sequence, as far as the block table reaches
};

// The request, or false (skipped): its query tokens are not inside [0,
// num_tokens), or more than max_query_len.
__device__ __forceinline__ bool request_of(const PerHeadAttentionArgs& a, int b, Request& r) {
  const int32_t q0 = load_global(a.query_start + b), q1 = load_global(a.query_start + b + 1);
  const int32_t len = max(0, load_global(a.seq_lens + b));
  r.token0 = q0;
  r.tokens = q1 - q0;
  r.first_pos = static_cast<int64_t>(len) - r.tokens;
  r.len = min(len, a.table_positions);
  r.cut = r.len < len;
  return q0 >= 0 && q1 >= q0 && q1 <= a.num_tokens && static_cast<int64_t>(q1) - q0 <= a.max_query_len;
}

// The keys that some token in [t0, t1] of the request sees.
template <int kStep>
__device__ __forceinline__ Keys<kStep> keys_of(const PerHeadAttentionArgs& a, const Request& r, int32_t t0, int32_t t1) {
  Keys<kStep> k;
  if (a.tree_mask != nullptr) {
    k.lo = k.sinks = 0;
    k.hi = r.len;
  } else {
    const int64_t p0 = r.first_pos + t0, p1 = r.first_pos + t1;
    k.hi = static_cast<int32_t>(min(static_cast<int64_t>(r.len), max(int64_t{0}, p1 + 1)));
    k.lo = a.window > 0 ? static_cast<int32_t>(min(static_cast<int64_t>(k.hi), max(int64_t{0}, p0 - a.window + 1))) : 0;
    k.sinks = min(a.num_sinks, k.lo);
  }
  k.sink_steps = (k.sinks + kStep - 1) / kStep;
  k.steps = k.sink_steps + (k.hi - k.lo + kStep - 1) / kStep;
  return k;
}

// The steps [s0, s1) of range `split` of a block of query rows: equal shares
// of the block's steps where its ranges run as a cluster (they wait for one
// another), else ranges of split_keys keys, of which the last takes the rest
// (ranges of equal length, whatever their sequence's, spread evenly over the GPU).
template <int kStep>
__device__ __forceinline__ void range_of(const PerHeadAttentionArgs& a, const Keys<kStep>& keys, int32_t split,
                                         int32_t& s0, int32_t& s1) {
  s0 = 0;
  s1 = keys.steps;
  if (a.num_splits == 1) return;
  const int64_t per = a.cluster ? (static_cast<int64_t>(keys.steps) + a.num_splits - 1) / a.num_splits : a.split_keys / kStep;
  s0 = static_cast<int32_t>(min(static_cast<int64_t>(keys.steps), split * per));
  if (split < a.num_splits - 1) s1 = static_cast<int32_t>(min(static_cast<int64_t>(keys.steps), (split + 1) * per));
}

// Range, row block and key head of a CTA.  Of the ranges of a cluster the
// number varies fastest; else the heads do, so that a token's heads,
// neighbours in an NHD page, are read at about the same time.
struct Place {
  uint32_t head;
  int32_t row_block, split;
};
__device__ __forceinline__ Place place_of(const PerHeadAttentionArgs& a, int32_t row_blocks) {
  uint32_t x = blockIdx.x;
  Place p;
  if (a.cluster) {
    p.split = static_cast<int32_t>(x % a.num_splits);
    x /= a.num_splits;
  }
  p.head = x % a.num_kv_heads;
  x /= a.num_kv_heads;
  p.row_block = static_cast<int32_t>(x % row_blocks);
  if (!a.cluster) p.split = static_cast<int32_t>(x / row_blocks);
  return p;
}

// Token and head of query row `flat` of a request and key head.
struct RowAt {
  int64_t token;
  int32_t head;
};
__device__ __forceinline__ RowAt row_at(const PerHeadAttentionArgs& a, const Request& r, uint32_t kv_head, uint32_t flat) {
  const uint32_t tk = a.group_div.div(flat);
  return {r.token0 + tk, static_cast<int32_t>(kv_head * a.group + (flat - tk * a.group))};
}

}  // namespace
}  // namespace kvq
