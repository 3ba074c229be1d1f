// kvq_fp8_gather.cuh -- which of a request's keys the gather of the e4m3 cache
// brings into the workspace, and where: the kernel that writes them and the
// attention that reads them use the same plan.
#pragma once

#include "kvq_dependent.cuh"
#include "kvq_launch.h"

namespace kvq {
namespace {

// The first key that a window lets a query at `position` see (window <= 0:
// none).  Negative positions, of padding, less a window may pass 32 bits.
__device__ __forceinline__ int32_t first_seen(int32_t position, int32_t window) {
  return window <= 0 || position < window ? 0 : position - window + 1;
}

// The request's rows of the workspace: the keys [0, sinks) that stay visible,
// then [lo, len), the ones that some of its queries may see.
struct GatherPlan {
  int32_t token0, n;           // its query tokens
  int32_t first;               // position of the first one (may be negative)
  int32_t len;                 // its keys, as far as the block table reaches
  bool cut;                    // there are more
  int32_t lo, sinks;
};
// false: the request is skipped (its tokens are not inside [0, num_tokens), or
// more than max_query_len, or its keys more than the workspace's rows).
__device__ __forceinline__ bool gather_plan(const CachedArgs& c, const int32_t* query_start, int64_t num_tokens,
                                            int32_t max_query_len, int32_t window, int32_t num_sinks, uint32_t b,
                                            GatherPlan& p) {
  const int32_t q0 = load_global(query_start + b), q1 = load_global(query_start + b + 1);
  const int32_t len = max(0, load_global(c.seq_lens + b));
  const int64_t n = static_cast<int64_t>(q1) - q0;
  if (q0 < 0 || n < 0 || q1 > num_tokens || n > max_query_len) return false;
  p.token0 = q0;
  p.n = static_cast<int32_t>(n);
  p.first = len - p.n;
  p.len = min(len, c.table_positions);
  p.cut = p.len < len;
  p.lo = min(p.len, first_seen(p.first, window));
  p.sinks = min(num_sinks, p.lo);
  return p.len - p.lo + p.sinks <= c.rows;
}

}  // namespace
}  // namespace kvq
