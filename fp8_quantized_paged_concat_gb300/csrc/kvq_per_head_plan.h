// kvq_per_head_plan.h -- which kernel, row block and key ranges a call of the
// per-head attention runs with: host arithmetic on the call's sizes, shared by
// the launcher and the default number of ranges, without CUDA.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kvq.h"

namespace kvq {

// CTAs of the few-row kernel that share an SM (its launch bounds).
constexpr int64_t resident_ctas(int32_t head_size, int64_t block) { return head_size == 256 ? 2 : block == 16 ? 3 : 4; }

// Rows per block of the few-row kernel.  16 rows share a decoded key where
// such blocks fill the GPU (128 requests x 2048 keys, head size 128, 16 rows:
// 111 us against 126 with two blocks of 8; 32 rows: 183 against 230); a
// smaller call is short of CTAs, and blocks of 8 halve its chain (one request
// x 1024 keys, 16 rows: 12.9 against 15.0 us; 16384 keys: 23 against 31).
// D = 256 has no registers for 16.
inline int64_t few_rows(int64_t rows, int64_t groups, int32_t head_size, int64_t splits, int sms) {
  return rows > 8 && head_size != 256 && (rows + 15) / 16 * groups * splits >= resident_ctas(head_size, 16) * int64_t{sms}
             ? 16 : 8;
}

// The most rows per request and key head that go to the few-row kernel, which
// decodes every key once per block of rows; above, the tensor memory kernel
// decodes it once.  us of the one and the other, 128 requests x 2048 keys x 8
// key heads (4 at D = 256):
//   D =  64: 48 rows 169 / 218, 64 rows 214 / 220, 96 rows 314 / 224
//   D = 128: 24 rows 181 / 232, 32 rows 183 / 234, 48 rows 265 / 240
//   D = 256: 16 rows 144 / 187, 24 rows 199 / 189, 32 rows 251 / 189
inline int64_t most_few_rows(int32_t head_size) { return head_size == 64 ? 64 : head_size == 128 ? 32 : 16; }

// Rows per block of the tensor memory kernel: one row tile, or two that share
// a decoded key (32 requests of 1024 keys x 256 rows, head size 128: 70 us
// against 99 with blocks of 128; D = 256 has tensor memory for one).
inline int64_t per_head_prefill_rows(int64_t rows, int32_t head_size) { return rows <= 128 || head_size == 256 ? 128 : 256; }

// Rows per block of the kernel that a call runs.
inline int64_t per_head_block(int64_t rows, int64_t groups, int32_t head_size, int64_t splits, bool cluster, int sms) {
  return !cluster && rows > most_few_rows(head_size) ? per_head_prefill_rows(rows, head_size)
                                                     : few_rows(rows, groups, head_size, splits, sms);
}

// The default key ranges per block of rows, whether they join through a
// workspace, and the block that they are sized for.
struct PerHeadRanges {
  int32_t splits;
  bool workspace;
  int64_t block;
};
inline PerHeadRanges per_head_default_ranges(int64_t max_query_len, int64_t group, int64_t num_kv_heads,
                                             int32_t head_size, int64_t batch_size, int64_t max_seq_len,
                                             int64_t window, int64_t num_sinks, int sms) {
  const int64_t rows = max_query_len * group, groups = num_kv_heads * batch_size;
  const bool windowed = window > 0 && window < max_seq_len;
  const int64_t keys =
      windowed ? std::min<int64_t>(max_seq_len, window + std::min<int64_t>(max_query_len, 256) + num_sinks) : max_seq_len;
  const bool few = rows <= most_few_rows(head_size);
  const bool ragged = !windowed && keys >= 4096 && batch_size > 1;   // long contexts, whose lengths may differ
  // A small call's ranges run as clusters of the few-row kernel: no second
  // launch.  Where the GPU has room for many more ranges than a cluster takes,
  // that pays for fewer keys (head size 128, us of a cluster of 8 and of 16
  // ranges through a workspace: one request, 8 key heads, 2048 keys 7.0 / 7.1,
  // 4096 keys 8.6 / 7.9, 8000 keys 10.9 / 9.0; four requests, room for 19,
  // 4096 keys 10.6 / 13.2, 8000 keys 14.3 / 15.4), and so it is where only two
  // CTAs share an SM (head size 256, four requests, 4 key heads: 2048 keys 12.6 /
  // 13.5, 4096 keys 16.0 / 15.6, 8000 keys 22.2 / 17.4).
  if (rows <= KVQ_PER_HEAD_CLUSTER_ROWS) {
    constexpr int64_t kMax = KVQ_PER_HEAD_CLUSTER_SPLITS, kLeast = 128;       // a step per warp
    const int64_t blocks = (rows + 7) / 8 * groups, places = resident_ctas(head_size, 8) * int64_t{sms};
    const bool long_small = ragged && 8 * blocks >= places;
    const int64_t room = places / blocks, n = std::min<int64_t>(keys / kLeast, room);
    if (!long_small && n > 1 && (n <= kMax || keys <= kMax * (room >= 4 * kMax || head_size == 256 ? 320 : 1024)))
      return {static_cast<int32_t>(std::min(n, kMax)), false, 8};
  }
  // between 1 and the most, and no more than the ranges of whole 128-key steps come to
  const auto whole = [&](int64_t n) {
    n = std::max<int64_t>(1, std::min<int64_t>(KVQ_PER_HEAD_MAX_SPLITS, n));
    const int64_t steps = (keys + 127) / 128, per = (steps + n - 1) / n;
    return (steps + per - 1) / per;
  };
  int64_t block = few ? few_rows(rows, groups, head_size, 1, sms) : per_head_prefill_rows(rows, head_size);
  const auto blocks = [&] { return (rows + block - 1) / block * groups; };
  const auto places = [&] { return (few ? resident_ctas(head_size, block) : 1) * int64_t{sms}; };
  int64_t n;
  if (ragged && 8 * blocks() >= places()) {
    // Several ranges to a CTA's place even the lengths out.  The few-row kernel
    // in blocks of 8: six, or two where there are more blocks than places (32
    // requests of 7k to 34k keys, 4 rows: 161 us; one range per place 217; equal
    // lengths would do with one, 4 to 20 % faster then).  In blocks of 16, which
    // such a call runs with wherever its ranges then fill the GPU: four (7k to
    // 34k keys: 16 requests, 8 key heads of 128, 32 rows: 232 us, three 253, and
    // 285 in blocks of 8; 64 requests, 2 key heads of 128, 16 rows: 132, three
    // 126, one 144, and 158; 64 requests, 8 key heads of 64, 12 rows: 259, three
    // 269, two 300, and 359 to 386).  The tensor memory
    // kernel, whose ranges cost more to start: three (32 requests x 8192 keys x
    // 48 rows at D = 256: 203 us, six 232), or six where there are more blocks
    // than places (32 trees of 64 drafts behind 7k to 34k keys: 611 us, three
    // 655, one 795).
    const auto ranges = [&](int64_t per_place) {
      return whole(std::min<int64_t>(keys / 1024, (per_place * places() + blocks() - 1) / blocks()));
    };
    if (few && rows > 8 && head_size != 256) {
      block = 16;
      n = ranges(4);
      if (few_rows(rows, groups, head_size, n, sms) != 16) block = 8;
    }
    if (block != 16) n = ranges(few == (blocks() >= places()) ? (few ? 2 : 3) : 6);
  } else {
    // As many as the call is short of CTAs, of at least 256 keys in the tensor
    // memory kernel.  In the few-row kernel a range costs keys / n steps and the
    // join n rows: their sum is least where n grows with the root of the keys
    // (one request, 8 key heads of 128: 8000 keys in 16 ranges 9.0 us, 32 9.4, 64
    // 11.5; 12000 keys 10.3, 10.6, 12.4; 65536 keys 46, 37, 33).
    n = whole(std::min<int64_t>(few ? static_cast<int64_t>(std::sqrt(keys / 16.0)) : keys / 256, places() / blocks()));
  }
  return {static_cast<int32_t>(n), n > 1, block};
}

}  // namespace kvq
