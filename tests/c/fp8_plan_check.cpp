// For calls over the e4m3 cache, over the whole range of sizes: the default key
// ranges are sized for the block of query rows that the call then runs with,
// stay within the entry points' limits, and a call that gathers its entries has
// the rows for it and room for every key that it may see.
#include <cstdio>

#include "kvq_per_head_plan.h"

int main() {
  long long calls = 0, gathers = 0, other_block = 0, out_of_limits = 0, no_room = 0;
  for (int sms : {152, 148, 132})
    for (int head_size : {64, 128, 256})
      for (int kv_heads : {1, 2, 3, 8, 16})
        for (int group : {1, 2, 3, 4, 7, 8, 16, 130})
          for (int query : {1, 2, 3, 4, 5, 8, 9, 16, 33, 64, 300, 4096})
            for (int batch : {1, 2, 3, 5, 6, 8, 13, 16, 31, 32, 57, 64, 128, 512})
              for (int keys : {1, 100, 1024, 4095, 4096, 5000, 9000, 16384, 34000, 131072, 1 << 20})
                for (int window : {0, 333, 8192}) {
                  const kvq::PerHeadRanges r =
                      kvq::per_head_default_ranges(query, group, kv_heads, head_size, batch, keys, window, 4, sms, true);
                  const long long rows = static_cast<long long>(query) * group;
                  const bool cluster = r.splits > 1 && !r.workspace, gather = r.splits == 1 && r.workspace;
                  ++calls;
                  if (r.splits < 1 || r.splits > KVQ_PER_HEAD_MAX_SPLITS ||
                      (gather && rows <= kvq::most_few_rows(head_size, true)) ||
                      (cluster && (r.splits > KVQ_PER_HEAD_CLUSTER_SPLITS || rows > KVQ_PER_HEAD_CLUSTER_ROWS)))
                    ++out_of_limits;
                  if (gather) {
                    ++gathers;
                    // a query sees its window and the sinks; the call's queries are one after the other
                    const long long held = kvq::fp8_gather_rows(query, keys, window, 4);
                    const long long seen = window > 0 && window + query - 1 + 4 < keys ? window + query - 1 + 4 : keys;
                    if (held < seen || held % 64 != 0 ||
                        kvq::fp8_gather_bytes(held, kv_heads, head_size, batch) <
                            batch * held * (4LL * kv_heads * head_size) + batch * held / 8 + 8)
                      ++no_room;
                  }
                  if (r.splits == 1) continue;
                  if (kvq::per_head_block(rows, static_cast<long long>(kv_heads) * batch, head_size, r.splits, cluster, sms,
                                          true) != r.block)
                    ++other_block;
                }
  std::printf("calls %lld, gathers %lld, other block %lld, out of limits %lld, no room %lld\n", calls, gathers, other_block,
              out_of_limits, no_room);
  return other_block + out_of_limits + no_room != 0;
}
