// For calls over the e4m3 cache whose default is to gather their entries, over
// the whole range of sizes: one request's fit into the room that the default
// counts on, as many at a time as the call then takes are the most that do, and
// a batch that goes through in rounds fills the GPU in each of them.  And a
// launch of any size, into workspaces of any size, has fewer than 2^31 rows and at
// most 2^25 block numbers.  And single tokens' blocks are cut into two ranges for the
// sake of a short last wave only.
#include <cstdio>

#include "kvq_per_head_plan.h"

int main() {
  long long gathers = 0, rounds = 0, no_room = 0, not_most = 0, idle = 0, unlike = 0;
  const long long room = KVQ_FP8_GATHER_BYTES;
  for (int sms : {152, 148, 132})
    for (int head_size : {64, 128, 256})
      for (int kv_heads : {1, 2, 3, 8, 16})
        for (int group : {1, 3, 4, 8, 16, 130})
          for (int query : {1, 5, 33, 64, 128, 300, 640, 4096})
            for (int batch : {1, 2, 3, 5, 8, 13, 32, 64, 128, 512, 4096})
              for (int keys : {1, 1024, 9000, 34000, 131072, 300000, 1 << 20, 1 << 30})
                for (int window : {0, 333, 8192}) {
                  const kvq::PerHeadRanges r =
                      kvq::per_head_default_ranges(query, group, kv_heads, head_size, batch, keys, window, 4, sms, true);
                  if (r.splits != 1 || !r.workspace) continue;
                  ++gathers;
                  const long long held = kvq::fp8_gather_rows(query, keys, window, 4);
                  const long long n = kvq::fp8_gather_at_once(held, kv_heads, head_size, batch, room);
                  if (n < 1 || n > batch || kvq::fp8_gather_bytes(held, kv_heads, head_size, n) > room) ++no_room;
                  if (n < batch && kvq::fp8_gather_bytes(held, kv_heads, head_size, n + 1) <= room) ++not_most;
                  const long long rows = 1LL * query * group, block = kvq::per_head_prefill_rows(rows, head_size);
                  const long long each = (rows + block - 1) / block * kv_heads;
                  if (n == batch) {
                    if (4 * each * n < 3 * sms) ++idle;
                    continue;
                  }
                  ++rounds;
                  // no round's blocks leave more than half of the GPU idle on average, and the rows pay for the gather
                  long long waves = 0;
                  for (long long b = 0; b < batch; b += n) waves += ((b + n < batch ? n : batch - b) * each + sms - 1) / sms;
                  if (rows < 1024 || 2 * waves > 3 * ((batch * each + sms - 1) / sms)) ++idle;
                  // the same rows as a batch that fits gather too
                  if (!kvq::fp8_default_gathers(query, group, kv_heads, head_size, batch, 1, 0, 4, sms) &&
                      kvq::fp8_gather_at_once(64, kv_heads, head_size, batch, room) == batch)
                    ++unlike;
                }
  // 128 query rows to a block, of whole tokens where a token's rows are fewer
  long long large = 0;
  for (long long group : {1, 2, 3, 4, 7, 8, 16, 43, 64, 65, 127, 128, 129, 130, 500})
    for (long long kv_heads : {1, 2, 3, 8, 128})
      for (long long query : {1LL, 25LL, 300LL, 4096LL, 65536LL, 1LL << 20, (1LL << 31) - 1})
        for (long long rows : {64LL, 4096LL, 1LL << 20, (1LL << 31) - 256}) {
          if (query * group * kv_heads >= 1LL << 31) continue;
          const long long tokens = group < 128 ? 128 / group : 1, chunks = (group + 127) / 128;
          const long long blocks = (query * chunks + tokens - 1) / tokens * kv_heads;
          const long long n = kvq::fp8_gather_most(rows, blocks);
          if (n < 1 || n * rows > (1LL << 31) - 256 || n * blocks > 1LL << 25) ++large;
        }
  // sizes that make no call are answered all the same
  for (int head_size : {0, -1, -128})
    if (kvq::fp8_gather_at_once(64, 8, head_size, 4, room) != 0 ||
        kvq::per_head_default_ranges(4096, 4, 8, head_size, 64, 4096, 0, 0, 152, true).splits < 1)
      ++large;
  long long full = 0, cut = 0;
  for (int batch = 1; batch < 400; ++batch)
    for (int keys : {1100, 2047, 2500, 4000})
      for (int sms : {152, 148}) {
        const kvq::PerHeadRanges r = kvq::per_head_default_ranges(1, 4, 8, 128, batch, keys, 0, 0, sms, true);
        const int places = 3 * sms, last = 8 * batch % places;
        if (8 * batch < places) continue;
        if (r.splits > 1) ++cut;
        if (r.splits > 1 && (keys < 2048 || 3 * last > places)) ++full;
      }
  std::printf("full last waves cut %lld of %lld, large %lld, gathers %lld, rounds %lld, no room %lld, not most %lld, idle %lld, unlike %lld\n", full, cut, large, gathers, rounds, no_room,
              not_most, idle, unlike);
  return (cut == 0) + full + large + no_room + not_most + idle + unlike != 0 || gathers == 0 || rounds == 0;
}
