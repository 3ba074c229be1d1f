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
// Bound: latency, of the chain from the request's lengths over its accepted
// list and the block table to the entries (26 MB move in the largest measured
// call), once per wave of CTAs.  So a CTA goes down that chain once, for one
// side and as many heads of a request as its threads hold, and then moves
// several layers' entries: a thread keeps kUnits units of kLayers layers in
// registers between its loads, all issued together, and its stores.  64
// requests x 32 layers of 8 heads: 13 us, in 1408 CTAs of 3 layers, three of
// which share an SM (74 registers a thread), so three waves (one CTA per layer
// and head: 80 us).
#include <algorithm>

#include "kvq_dependent.cuh"
#include "kvq_device.cuh"
#include "kvq_launch.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;                    // units per thread and chunk
constexpr int kLayers = 4;                   // layers in flight

// Page in column `col` of request b's table, or -1.
__device__ __forceinline__ int64_t page_of(const CompactArgs& a, int b, uint32_t col) {
  if (col >= static_cast<uint32_t>(a.block_table_width)) return -1;
  const int32_t id = load_global(a.block_table + b * a.block_table_stride + col);
  return id >= 0 && id < a.num_pages ? id : -1;
}

template <int kBytes>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };

// Unit: kDataBytes data bytes, or kScaleBytes scale bytes.  heads: of a CTA.
template <int kDataBytes, int kScaleBytes>
__global__ void __launch_bounds__(kThreads) compact_drafts_kernel(const CompactArgs a, int heads, int layers_per_cta) {
  using Data = typename Word<kDataBytes>::type;
  wait_for_previous();
  allow_dependents();
  const int b = blockIdx.x, side = blockIdx.y & 1;
  const int head0 = static_cast<int>(blockIdx.y >> 1) * heads;
  const int layer0 = blockIdx.z * layers_per_cta, layer1 = min(a.num_layers, layer0 + layers_per_cta);
  const bool first = blockIdx.y == 0 && blockIdx.z == 0;
  const int32_t q0 = load_global(a.query_start + b), q1 = load_global(a.query_start + b + 1);
  const int64_t n = static_cast<int64_t>(q1) - q0, len = load_global(a.seq_lens + b);
  const int32_t m = load_global(a.accepted_lens + b);
  if (m == 0) return;
  if (n < 0 || len < n) {                                  // uniform over the CTA
    if (first && threadIdx.x == 0) report(a.status, KVQ_STATUS_BAD_BATCH);
    return;
  }
  const uint32_t base = static_cast<uint32_t>(len - n);
  const int32_t* acc = a.accepted + b * a.accepted_stride;
  bool bad = m < 0 || m > a.max_accepted;
  if (!bad) {
    for (int i = threadIdx.x; i < m; i += kThreads) {
      const int32_t x = load_global(acc + i);
      if (x < 0 || x >= n || (i > 0 && x <= load_global(acc + i - 1))) bad = true;
    }
  }
  if (__syncthreads_or(bad)) {                             // a malformed list: the request is left as it is
    if (first && threadIdx.x == 0) report(a.status, KVQ_STATUS_BAD_INDEX);
    return;
  }
  const int groups = a.head_size / kGroup;
  const int data_units = a.head_size / 2 / kDataBytes, row_units = data_units + groups / kScaleBytes;
  const int my_heads = min(heads, a.num_kv_heads - head0), move_units = my_heads * row_units;
  const int64_t scales = static_cast<int64_t>(a.block_size) * a.num_kv_heads * (a.head_size / 2);
  const int64_t region = scales + static_cast<int64_t>(a.block_size) * a.num_kv_heads * groups;
  uint8_t* cache = a.cache + side * region;
  const int moves = max(1, kThreads * kUnits / move_units);      // per chunk (the host sees to move_units)
  for (int i0 = 0; i0 < m; i0 += moves) {
    const int units = min(moves, m - i0) * move_units;
    int64_t from[kUnits], to[kUnits];                      // offsets in a layer, -1: nothing to move
    bool is_data[kUnits];
    bool missing = false;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = threadIdx.x + j * kThreads;
      to[j] = -1;
      if (u >= units) continue;
      const int i = i0 + u / move_units, in_move = u % move_units;
      const int head = head0 + in_move / row_units, w = in_move % row_units;
      const uint32_t from_p = base + static_cast<uint32_t>(load_global(acc + i)), to_p = base + i;   // below seq_lens[b]
      if (from_p == to_p) continue;
      const uint32_t from_col = a.block_div.div(from_p), to_col = a.block_div.div(to_p);
      const int64_t from_page = page_of(a, b, from_col), to_page = page_of(a, b, to_col);
      if (from_page < 0 || to_page < 0) {
        missing = true;
        continue;
      }
      // row of (offset, head) in its page's side region
      const int64_t off0 = from_p - from_col * static_cast<uint32_t>(a.block_size);
      const int64_t off1 = to_p - to_col * static_cast<uint32_t>(a.block_size);
      const int64_t row0 = a.layout == KVQ_LAYOUT_HND ? static_cast<int64_t>(head) * a.block_size + off0
                                                      : off0 * a.num_kv_heads + head;
      const int64_t row1 = row0 + (off1 - off0) * (a.layout == KVQ_LAYOUT_HND ? 1 : a.num_kv_heads);
      is_data[j] = w < data_units;
      const int64_t pitch = is_data[j] ? a.head_size / 2 : groups;
      const int64_t in_row = is_data[j] ? kDataBytes * w : scales + kScaleBytes * (w - data_units);
      from[j] = from_page * 2 * region + row0 * pitch + in_row;
      to[j] = to_page * 2 * region + row1 * pitch + in_row;
    }
    if (missing && first) report(a.status, KVQ_STATUS_BAD_INDEX);
    for (int l0 = layer0; l0 < layer1; l0 += kLayers) {
      Data v[kUnits][kLayers];
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
#pragma unroll
        for (int l = 0; l < kLayers; ++l) {
          if (to[j] < 0 || l0 + l >= layer1) continue;
          const uint8_t* src = cache + (l0 + l) * a.layer_stride + from[j];
          if (is_data[j])
            v[j][l] = *reinterpret_cast<const Data*>(src);
          else if constexpr (kScaleBytes == 4)
            v[j][l].x = *reinterpret_cast<const uint32_t*>(src);
          else
            v[j][l].x = *src;
        }
      }
      __syncthreads();                                     // every read of the chunk in these layers is done
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
#pragma unroll
        for (int l = 0; l < kLayers; ++l) {
          if (to[j] < 0 || l0 + l >= layer1) continue;
          uint8_t* dst = cache + (l0 + l) * a.layer_stride + to[j];
          if (is_data[j])
            *reinterpret_cast<Data*>(dst) = v[j][l];
          else if constexpr (kScaleBytes == 4)
            *reinterpret_cast<uint32_t*>(dst) = v[j][l].x;
          else
            *dst = static_cast<uint8_t>(v[j][l].x);
        }
      }
    }
  }
}

template <int kDataBytes, int kScaleBytes>
cudaError_t launch(const CompactArgs& a, int num_sms, cudaStream_t stream) {
  const int groups = a.head_size / kGroup;
  const int row_units = a.head_size / 2 / kDataBytes + groups / kScaleBytes;   // at most 192 (head_size <= 1024)
  const int heads = std::max(1, std::min(a.num_kv_heads, kThreads * kUnits / row_units));
  const int64_t chunks = (a.num_kv_heads + heads - 1) / heads;
  // layers of a CTA: as many as leave about eight CTAs to each SM of the whole
  // grid, of which three run at a time
  const int64_t ctas = static_cast<int64_t>(a.batch_size) * 2 * chunks * a.num_layers;
  const int per_cta = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, ctas / (8 * num_sms))));
  const dim3 grid(static_cast<unsigned>(a.batch_size), static_cast<unsigned>(2 * chunks),
                  static_cast<unsigned>((a.num_layers + per_cta - 1) / per_cta));
  return launch_dependent(compact_drafts_kernel<kDataBytes, kScaleBytes>, grid, kThreads, 0, 1, stream, a, heads, per_cta);
}

}  // namespace

cudaError_t launch_compact_drafts(const CompactArgs& a, int num_sms, cudaStream_t stream) {
  // data in 16 bytes and scales in words where the rows and regions allow it
  // (a region is a multiple of 8 bytes: host check)
  const int64_t region = static_cast<int64_t>(a.block_size) * a.num_kv_heads * (a.head_size / 2 + a.head_size / kGroup);
  const bool wide = a.head_size % 32 == 0 && region % 16 == 0;
  if ((a.head_size / kGroup) % 4 == 0) return wide ? launch<16, 4>(a, num_sms, stream) : launch<8, 4>(a, num_sms, stream);
  return wide ? launch<16, 1>(a, num_sms, stream) : launch<8, 1>(a, num_sms, stream);
}

}  // namespace kvq
