// kvq_fp8_gather.cu -- the e4m3 cache's entries of the keys that a call's
// requests see, as bf16 rows of a workspace: exact, an e4m3 value has four
// significant bits and the page scales are powers of two.  For chunks of many
// query rows, whose attention reads every key many times: it decodes each once,
// where the attention over the pages decodes it for every 256 rows (128 at head
// size 256).
//
// Bound: HBM (a byte read and two written for each value).  One warp takes 32
// rows and every fourth (head, side): lane l looks up row l's page once; then
// D / 16 lanes take a row, twice 8 values each, so that loads and stores of a
// warp fill whole sectors (16 neighbouring values to a lane: 38 us for the 27
// below), every row's load of a (head, side) under way at once.  Measured: 24139
// entries of 8 heads of 128, 148 MB: 27 us = 5.5 TB/s.
#include "kvq_fp8_gather.cuh"
#include "kvq_per_head_attention.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) fp8_gather_kernel(const Fp8GatherArgs a) {
  constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes, kPasses = D == 64 ? 4 : 8;   // rows of a load, loads at once
  constexpr int kRounds = 32 / (kAtOnce * kPasses);
  wait_for_previous();
  allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b = blockIdx.y;
  GatherPlan plan;
  if (!gather_plan(a.cached, a.query_start, a.num_tokens, a.max_query_len, a.window, a.num_sinks, b, plan)) return;
  if (plan.n == 0) return;
  const int32_t r0 = blockIdx.x * 32, rows = plan.sinks + plan.len - plan.lo;
  if (blockIdx.x == 0 && threadIdx.x == 0 && plan.cut) report(a.status, KVQ_STATUS_BAD_INDEX);
  // lane l: row r0 + l
  const int32_t r = r0 + lane;
  const uint32_t p = static_cast<uint32_t>(r < plan.sinks ? r : r - plan.sinks + plan.lo);
  const uint32_t col = a.block_div.div(p);
  int32_t id = -1;
  if (r < rows) id = load_global(a.block_table + b * a.block_table_stride + col);   // (p < len <= the table's positions)
  const bool ok = id >= 0 && id < a.num_pages;
  if (r < rows && !ok) report(a.status, KVQ_STATUS_BAD_INDEX);
  const uint32_t there = __ballot_sync(kFull, ok);
  if (warp == 0 && lane == 0)
    a.there[(static_cast<int64_t>(b) * a.cached.rows + r0) >> 5] = there;
  if (r0 >= rows) return;
  const uint32_t row = (p - col * static_cast<uint32_t>(a.block_size)) * static_cast<uint32_t>(a.row_offset);
  const int sub = lane / kLanes, c = lane % kLanes;
  const int64_t out_row0 = static_cast<int64_t>(b) * a.cached.rows + r0;
#pragma unroll 1
  for (int round = 0; round < kRounds; ++round) {
    // what a pass needs of its row
    uint32_t page[kPasses], page_row[kPasses];
    const int row_in = round * kAtOnce * kPasses + sub;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int from = i * kAtOnce + row_in;
      page[i] = __shfl_sync(kFull, ok ? static_cast<uint32_t>(id) : 0u, from);
      page_row[i] = __shfl_sync(kFull, row, from);
    }
    for (int32_t hs = warp; hs < 2 * a.num_kv_heads; hs += kWarps) {
      const int32_t side = hs & 1, head = hs >> 1;
      uint2 w[kPasses][2];                          // values 8 c on, and D / 2 + 8 c on
      uint32_t e[kPasses];
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int from = i * kAtOnce + row_in;
        w[i][0] = w[i][1] = make_uint2(0, 0);
        e[i] = KVQ_FP8_SCALE_BIAS;
        if ((there >> from) & 1) {
          const uint8_t* region = at_offset(a.cache + (side ? a.region : 0), page[i], 2 * a.region);
          const uint2* x = reinterpret_cast<const uint2*>(at_offset(region, page_row[i] + head * a.row_head, D)) + c;
          w[i][0] = load_global(x);
          w[i][1] = load_global(x + kLanes);
          e[i] = load_global(a.page_scales + (static_cast<uint64_t>(page[i]) * 2 + side) * a.num_kv_heads + head);
        }
      }
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(side ? a.v : a.k);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int from = i * kAtOnce + row_in;
        if (r0 + from >= rows) continue;
        const float f = __uint_as_float(page_scale(e[i]) << 23);
        const uint32_t x[4] = {w[i][0].x, w[i][0].y, w[i][1].x, w[i][1].y};
        uint32_t y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 v = __half22float2(e4m3x2_to_half2(x[j >> 1] >> (16 * (j & 1))));
          y[j] = pack_bf16x2(v.x * f, v.y * f);
        }
        uint4* to = reinterpret_cast<uint4*>(out + ((out_row0 + from) * a.num_kv_heads + head) * D) + c;
        to[0] = make_uint4(y[0], y[1], y[2], y[3]);
        to[kLanes] = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
  }
}

template <int D>
cudaError_t launch(const Fp8GatherArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.cached.rows / 32), static_cast<unsigned>(a.batch_size));
  return launch_dependent(fp8_gather_kernel<D>, grid, kWarps * 32, 0, 1, stream, a);
}

}  // namespace

cudaError_t launch_fp8_gather(const Fp8GatherArgs& a, cudaStream_t stream) {
  switch (a.head_size) {
    case 64: return launch<64>(a, stream);
    case 128: return launch<128>(a, stream);
    default: return launch<256>(a, stream);
  }
}

}  // namespace kvq
