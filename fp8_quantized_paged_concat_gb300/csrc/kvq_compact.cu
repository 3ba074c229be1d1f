// kvq_compact.cu -- after a tree of drafted tokens was checked: the accepted
// drafts' entries in the per-head NVFP4 cache move to consecutive positions.
//
// Request b's drafts sit at positions base .. base + n - 1 (base = seq_lens[b]
// - n).  With its accepted draft numbers a_0 < a_1 < ..., the entry of
// position base + a_i moves to base + i, in every layer, side and head.
// Since the numbers increase, a_i >= i: a destination is never the source of
// a later move, so the moves are made in chunks, in order, and only inside a
// chunk must every read come before the first write.
//
// Bound: latency (a few KB per request and layer; 26 MB moved in the largest
// measured call).  One CTA per (request, layer, side, head chunk); a thread
// keeps up to kUnits units of a chunk in registers between its loads and its
// stores.
#include "kvq_device.cuh"
#include "kvq_launch.h"

namespace kvq {
namespace {

constexpr int kThreads = 128;
constexpr int kUnits = 4;                    // units per thread and chunk

// Row index of (offset, head) in its page's side region.
__device__ __forceinline__ int64_t row_of(const CompactArgs& a, uint32_t off, int head) {
  return a.layout == KVQ_LAYOUT_HND ? static_cast<int64_t>(head) * a.block_size + off
                                    : static_cast<int64_t>(off) * a.num_kv_heads + head;
}

// Page holding position p of request b, or -1.
__device__ __forceinline__ int64_t page_of(const CompactArgs& a, int b, int64_t p) {
  const int64_t col = p / a.block_size;
  if (p < 0 || col >= a.block_table_width) return -1;
  const int32_t id = __ldg(a.block_table + b * a.block_table_stride + col);
  return id >= 0 && id < a.num_pages ? id : -1;
}

// Unit: 8 data bytes, or one scale word (kScaleBytes).  Units of an entry's
// head row: head_size / 16 data units, then its scale words.
template <int kScaleBytes>
__global__ void __launch_bounds__(kThreads) compact_drafts_kernel(const CompactArgs a) {
  const int b = blockIdx.x, head = blockIdx.y;
  const int layer = blockIdx.z >> 1, side = blockIdx.z & 1;
  const bool first = head == 0 && blockIdx.z == 0;
  const int32_t q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
  const int64_t n = static_cast<int64_t>(q1) - q0, len = __ldg(a.seq_lens + b);
  const int32_t m = __ldg(a.accepted_lens + b);
  if (m == 0) return;
  if (n < 0 || len < n) {                                  // uniform over the CTA
    if (first && threadIdx.x == 0) report(a.status, KVQ_STATUS_BAD_BATCH);
    return;
  }
  const int64_t base = len - n;
  const int32_t* acc = a.accepted + b * a.accepted_stride;
  bool bad = m < 0 || m > a.max_accepted;
  if (!bad) {
    for (int i = threadIdx.x; i < m; i += kThreads) {
      const int32_t x = __ldg(acc + i);
      if (x < 0 || x >= n || (i > 0 && x <= __ldg(acc + i - 1))) bad = true;
    }
  }
  if (__syncthreads_or(bad)) {                             // a malformed list: the request is left as it is
    if (first && threadIdx.x == 0) report(a.status, KVQ_STATUS_BAD_INDEX);
    return;
  }
  const int groups = a.head_size / kGroup, words = groups / kScaleBytes, per_row = groups + words;
  const int64_t data_dim = a.head_size / 2;
  const int64_t scales = static_cast<int64_t>(a.block_size) * a.num_kv_heads * data_dim;
  const int64_t region = scales + static_cast<int64_t>(a.block_size) * a.num_kv_heads * groups;
  uint8_t* cache = a.cache + layer * a.layer_stride + side * region;
  const int rows = max(1, kThreads * kUnits / per_row);    // moves per chunk
  for (int i0 = 0; i0 < m; i0 += rows) {
    const int units = min(rows, m - i0) * per_row;
    uint2 v[kUnits];
    uint8_t* to[kUnits];
    bool missing = false;
    // (per_row can exceed what the threads hold at once only for head sizes
    // past kThreads * kUnits * 8; the host bounds head_size well below that)
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = threadIdx.x + j * kThreads;
      to[j] = nullptr;
      if (u >= units) continue;
      const int i = i0 + u / per_row, w = u % per_row;
      const int64_t from_p = base + __ldg(acc + i), to_p = base + i;
      if (from_p == to_p) continue;
      const int64_t from_page = page_of(a, b, from_p), to_page = page_of(a, b, to_p);
      if (from_page < 0 || to_page < 0) {
        missing = true;
        continue;
      }
      const int64_t from_row = row_of(a, static_cast<uint32_t>(from_p % a.block_size), head);
      const int64_t to_row = row_of(a, static_cast<uint32_t>(to_p % a.block_size), head);
      const uint8_t* src = cache + from_page * 2 * region;
      uint8_t* dst = cache + to_page * 2 * region;
      if (w < groups) {
        v[j] = *reinterpret_cast<const uint2*>(src + from_row * data_dim + 8 * w);
        to[j] = dst + to_row * data_dim + 8 * w;
      } else {
        const int64_t s = scales + kScaleBytes * (w - groups);
        if constexpr (kScaleBytes == 4)
          v[j].x = *reinterpret_cast<const uint32_t*>(src + s + from_row * groups);
        else
          v[j].x = src[s + from_row * groups];
        to[j] = dst + s + to_row * groups;
      }
    }
    if (missing && head == 0 && blockIdx.z == 0) report(a.status, KVQ_STATUS_BAD_INDEX);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      if (to[j] == nullptr) continue;
      const int w = (threadIdx.x + j * kThreads) % per_row;
      if (w < groups)
        st8(to[j], v[j]);
      else if constexpr (kScaleBytes == 4)
        st4(to[j], v[j].x);
      else
        *to[j] = static_cast<uint8_t>(v[j].x);
    }
  }
}

}  // namespace

cudaError_t launch_compact_drafts(const CompactArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.batch_size), static_cast<unsigned>(a.num_kv_heads),
                  static_cast<unsigned>(2 * a.num_layers));
  // scale rows are moved in words when they and the regions allow it
  if ((a.head_size / kGroup) % 4 == 0)
    compact_drafts_kernel<4><<<grid, kThreads, 0, stream>>>(a);
  else
    compact_drafts_kernel<1><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
