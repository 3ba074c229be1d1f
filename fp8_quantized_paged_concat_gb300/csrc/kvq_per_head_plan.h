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
// such blocks and their ranges fill the GPU (128 requests x 2048 keys, head
// size 128, 16 rows: 97 us against 117 with two blocks of 8; 32 rows: 173
// against 220); a smaller call is short of CTAs, and blocks of 8 halve its
// chain (one request x 1024 keys, 16 rows: 6.9 us against 8.8; with long
// contexts, whose ranges are many, blocks of 16 would be as good: 16384 keys
// 16.9 against 15.7).  D = 256 has no registers for 16.
inline int64_t few_rows(int64_t rows, int64_t groups, int32_t head_size, int64_t splits, int sms) {
  return rows > 8 && head_size != 256 && (rows + 15) / 16 * groups * splits >= resident_ctas(head_size, 16) * int64_t{sms}
             ? 16 : 8;
}

// The most rows per request and key head that go to the few-row kernel, which
// decodes every key once per block of rows; above, the tensor memory kernel
// decodes it once.  us of the one and the other, 128 requests x 2048 keys x 8
// key heads (4 at D = 256), unsplit:
//   D =  64: 48 rows 159 / 179, 64 rows 204 / 179, 96 rows 303 / 179
//   D = 128: 24 rows 171 / 193, 32 rows 173 / 193, 48 rows 253 / 193
//   D = 256: 16 rows 124 / 170, 24 rows 187 / 171, 32 rows 236 / 171
// (The limit at D = 64 was set when the tensor memory kernel took 220 there; a
// call this large is now past the crossing at 64 rows.)
inline int64_t most_few_rows(int32_t head_size) { return head_size == 64 ? 64 : head_size == 128 ? 32 : 16; }

// Rows per block of the tensor memory kernel: one row tile, or two that share
// a decoded key (32 requests of 1024 keys x 256 rows, head size 128: 41 us
// against 68 with blocks of 128; D = 256 has tensor memory for one).
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
  // ranges through a workspace: one request, 8 key heads, 2048 keys 6.2 / 6.4,
  // 4096 keys 7.9 / 7.2, 8000 keys 10.9 / 9.0; four requests, room for 19,
  // 4096 keys 10.0 / 11.8, 8000 keys 14.3 / 15.7), and so it is where only two
  // CTAs share an SM (head size 256, four requests, 4 key heads: 2048 keys 11.4 /
  // 11.9, 4096 keys 14.9 / 13.9, 8000 keys 22.2 / 17.7).
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
    // Several ranges to a CTA's place even the lengths out.
    // The few-row kernel in blocks of 8: six, or two where there are more blocks
    // than places (32 requests x 4 rows: 7k to 34k keys 157 us, one range per
    // place 175 to 239, unsplit 248; 16384 keys each 130, and 131 and 138, at
    // best 117 in 4 ranges.  128 requests: ragged 620, unsplit 705, in 4 ranges
    // 584; 8192 keys each 222, 217, 229: the lengths are not known here).
    // In blocks of 16, which such a call runs with wherever its ranges then fill
    // the GPU: four (7k to 34k keys: 16 requests, 8 key heads of 128, 32 rows:
    // 232 us, three 253, and 306 in blocks of 8; 64 requests, 2 key heads of 128,
    // 16 rows: 132, three 126, one 144, and 158; 64 requests, 8 key heads of 64,
    // 12 rows: 259, three 269, two 300, and 359).
    // The tensor memory kernel, whose ranges cost more to start: three (32
    // requests x 48 rows at D = 256: 8192 keys each 181 us, six 191, unsplit 152;
    // 7k to 34k keys 367, six 347, unsplit 594), or six where there are more
    // blocks than places (32 trees of 64 drafts, four ranges: behind 7k to 34k
    // keys 588, unsplit 665; behind 20000 each 535, unsplit 518).
    const auto ranges = [&](int64_t per_place) {
      return whole(std::min<int64_t>(keys / 1024, (per_place * places() + blocks() - 1) / blocks()));
    };
    if (few && rows > 8 && head_size != 256) {
      block = 16;
      n = ranges(4);
      if (few_rows(rows, groups, head_size, n, sms) != 16) block = 8;
    }
    if (block != 16) {
      const bool many = blocks() >= places();
      n = ranges(few ? (many ? 2 : 6) : (many ? 6 : 3));
    }
  } else {
    // As many as the call is short of CTAs, of at least 256 keys in the tensor
    // memory kernel.  In the few-row kernel a range costs keys / n steps and the
    // join n rows: their sum is least where n grows with the root of the keys
    // (one request, 8 key heads of 128: 8000 keys in 16 ranges 8.9 us, 32 9.6, 64
    // 11.6; 12000 keys 10.5, 10.7, 12.6; 65536 keys 30, 25, 26).
    n = whole(std::min<int64_t>(few ? static_cast<int64_t>(std::sqrt(keys / 16.0)) : keys / 256, places() / blocks()));
  }
  return {static_cast<int32_t>(n), n > 1, block};
}

}  // namespace kvq
