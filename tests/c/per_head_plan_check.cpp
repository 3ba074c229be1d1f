// For calls over the whole range of sizes: the default key ranges of the
// per-head attention are sized for the block of query rows that the call then
// runs with, and stay within the entry points' limits.
#include <cstdio>

#include "kvq_per_head_plan.h"

int main() {
  long long calls = 0, split = 0, other_block = 0, out_of_limits = 0;
  for (int sms : {152, 148, 132})
    for (int head_size : {64, 128, 256})
      for (int kv_heads : {1, 2, 3, 8, 16})
        for (int group : {1, 2, 3, 4, 7, 8, 16})
          for (int query : {1, 2, 3, 4, 5, 8, 9, 16, 33, 64, 300, 4096})
            for (int batch : {1, 2, 3, 5, 6, 8, 13, 16, 31, 32, 57, 64, 128, 512})
              for (int keys : {1, 100, 1024, 4095, 4096, 5000, 9000, 16384, 34000, 131072, 1 << 20})
                for (int window : {0, 333, 8192}) {
                  const kvq::PerHeadRanges r =
                      kvq::per_head_default_ranges(query, group, kv_heads, head_size, batch, keys, window, 4, sms);
                  const long long rows = static_cast<long long>(query) * group;
                  const bool cluster = r.splits > 1 && !r.workspace;
                  ++calls;
                  if (r.splits < 1 || r.splits > KVQ_PER_HEAD_MAX_SPLITS || (r.workspace && r.splits == 1) ||
                      (cluster && (r.splits > KVQ_PER_HEAD_CLUSTER_SPLITS || rows > KVQ_PER_HEAD_CLUSTER_ROWS)))
                    ++out_of_limits;
                  if (r.splits == 1) continue;
                  ++split;
                  const long long runs = kvq::per_head_block(rows, static_cast<long long>(kv_heads) * batch, head_size,
                                                             r.splits, cluster, sms);
                  if (runs != r.block && other_block++ < 5)
                    std::printf("head_size %d, %d key heads, %lld rows, %d requests x %d keys, %d SMs: %d ranges sized "
                                "for blocks of %lld, run with %lld\n",
                                head_size, kv_heads, rows, batch, keys, sms, r.splits, static_cast<long long>(r.block), runs);
                }
  std::printf("calls %lld, split %lld, other block %lld, out of limits %lld\n", calls, split, other_block, out_of_limits);
  return other_block + out_of_limits != 0;
}
