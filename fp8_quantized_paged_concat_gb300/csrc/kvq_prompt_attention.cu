// kvq_prompt_attention.cu -- causal attention over whole prompts: packed
// sequences of different lengths, grouped query heads, a sliding window and a
// few first tokens that stay visible.  For query row (token i, head h) of a
// sequence, over its tokens j <= i with window <= 0 or j > i - window or j <
// num_sinks, and key head h / group:
//   s_j = softmax_scale * (q . k_j),  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + ln sum_j exp(s_j - m).
// The products bound it: 4 D flops for each (row, visible key).
//
// Design: one CTA per SM (two where sequences fit one row tile, and head_size
// <= 128: 256 sequences of 30 tokens, 32 query heads of 128, 61 -> 48 us; where
// they take more, blocks of two tiles read their keys half as often: 16 x 1000
// tokens 133 us, 220 with one), which takes one item after the other: (block of
// 128 kTiles query rows, key head, sequence).  The grid has a CTA per item; one
// that runs takes over the next that has not started, whose keys and queries
// are copied while it finishes.  Long items come first.  The rows are (token,
// head) pairs of the sequence that share the key head, so that every tile of
// keys serves the whole group.
//   - tensor memory: O of row tile w in columns [D w, +D), behind them two score
//     buffers of kKeys columns for each row tile.  A buffer's weights P (bf16)
//     overwrite its first half.
//   - one warp per row tile issues its products, in the order S(0) S(1) [PV(0)
//     S(2)] [PV(1) S(3)] ... over the key tiles: while the weights of one are
//     computed, the products of the other row tile run.  The tensor core takes
//     them in that order, so that S(i + 2) needs no wait for the PV(i) that
//     reads its buffer.  (128-key tiles with one buffer per row tile, and one
//     warp for both: 1 x 16384 tokens 1574 us against 1250.)
//   - one warp has the copy engine land the query rows and the tiles of K and V
//     (tensor maps, 128-byte swizzle); a tile of query rows holds all of the
//     group's heads of as many whole tokens as it has room for.
//   - four softmax warps per row tile, one thread per row, one pass over the
//     scores: the weights are formed against the reference maximum of the tiles
//     before, without a maximum of their own; only when their sum shows that
//     one of them may exceed it by more than 2^24 is the tile's maximum taken,
//     the pass repeated and O rescaled.  (bf16 weights have fp32's range, so
//     that a reference far behind costs no precision.)
//   - a tile's copy may bring rows that no query sees: the next sequence's,
//     padding, or later tokens.  Their scores are replaced, and their values,
//     whose weight is 0, are made harmless in shared memory: rows past the
//     sequence are zeroed, and in tiles that some row does not see whole NaN
//     and infinities are (one or two warps look through them).
// Measured (32 query heads, 8 key heads; calls one after the other), and of
// 1947 TFLOP/s: D = 128, 1 x 16384 tokens 1330 to 1370 us = 1600 to 1650 TFLOP/s,
// 0.83, with the SM clock at 1665 MHz under the power cap (the first few calls on
// an idle GPU, at 2070 MHz, 1200 us = 1830); 4 x 4096 375 us = 1465, 0.75 (first 345);
// 16 x 1024 136 us = 1009, 0.52.  A pair of row tiles takes
// about 1330 clocks a key tile, of which the products take 1280 (S at 48 clocks
// per 16 dimensions, bound by shared memory, PV at 64 per 16 keys); an item
// costs some 4000 more, for its first and last tiles' masks and its output.
// D = 64: 1 x 16384 1086 us = 1012 TFLOP/s, where the chain from a tile's scores
// to its weights (1170 clocks) is longer than the products of both row tiles (2 x
// 384).  D = 256: 1 x 8192 770 us = 1430, one row tile, whose keys come from L2
// twice as often, into two stages.
// Every wait of a role on another role or on its products is bounded; on
// expiry the CTA records KVQ_STATUS_TIMEOUT, drains its copies and products,
// frees its tensor memory and leaves its rows unwritten.
#include <type_traits>

#include "kvq_fp8_gather.cuh"
#include "kvq_per_head_attention.cuh"
#include "kvq_tensor_map.h"

namespace kvq {
namespace {

constexpr float kMaxSum = 16777216.0f;            // 2^24: weights against a reference this far behind are still finite
constexpr int kSlots = 2;                         // work items known at once

template <int D, int kTiles>
struct Shape {
  static constexpr int kKeys = 64;                           // keys per tile
  static constexpr int kSoftmaxWarps = 4 * kTiles;
  static constexpr int kCopyWarp = kSoftmaxWarps, kProductWarp = kCopyWarp + 1, kProductWarps = kTiles;
  static constexpr int kCheckWarp = kProductWarp + kProductWarps, kCheckWarps = 3 - kTiles;
  static constexpr int kWarps = kCheckWarp + kCheckWarps;
  static constexpr int kThreads = 32 * kWarps;
  // One row tile leaves room for a second CTA on the SM (but for D = 256).
  static constexpr int kCtas = kTiles == 1 && D <= 128 ? 2 : 1;
  static constexpr uint32_t kTmemCols = 512 / kCtas, kSCol = kTmemCols / 2;
  // the registers of a thread at launch, split by role
  static constexpr bool kSplitRegs = D <= 128;
  static constexpr int kRegs = kCtas == 2 ? 128 : 168, kSoftmaxRegs = kCtas == 2 ? 168 : 208, kOtherRegs = 88;
  static_assert(!kSplitRegs || 32 * kSoftmaxWarps * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kRegs, "register split");
  static constexpr int kBlocks = D / 64;                     // 64-dimension blocks
  static constexpr int kStages = D == 256 || (D == 128 && kCtas == 2) ? 2 : 4;           // tiles of K, of V
  static constexpr int kAhead = 2;                           // scores before a tile's output
  // One row tile: a tile's output is issued before the keys of the scores behind
  // it are waited for, which with two stages come late (D = 256, 1 x 8192 tokens:
  // 845 us, 1137 the other way round), and keys are copied a tile before the
  // values, their stage being free earlier (774 us).  Two row tiles: the keys are
  // waited for before the weights, and the scores follow the output at once (D =
  // 128, 1 x 16384 tokens: 1200 us, 1373 the other way round; with keys copied
  // first 1225, and 16 x 1024 tokens 146 for 137).
  static constexpr bool kKeysLast = kTiles == 1;
  static constexpr int kKeysFirst = kTiles == 1 ? 1 : 0;     // tiles that keys are copied ahead of values
  static constexpr uint32_t kQBlock = 128 * 128;             // 64 dimensions of a row tile
  static constexpr uint32_t kQTile = kBlocks * kQBlock;
  static constexpr uint32_t kKBlock = kKeys * 128;           // 64 dimensions of a key tile
  static constexpr uint32_t kTileBytes = kBlocks * kKBlock;
  static constexpr uint32_t kK = kTiles * kQTile;
  static constexpr uint32_t kV = kK + kStages * kTileBytes;
  static constexpr uint32_t kOut = kV + kStages * kTileBytes;          // 4 KB of output rows per softmax warp
  static constexpr uint32_t kMisc = kOut + kSoftmaxWarps * 4096;
  // The tiles begin on a 1024-byte boundary; 512 bytes of barriers take what is left before or behind them.
  // At least 116 KB where a second CTA, which would wait for tensor memory, must not share the SM.
  static constexpr uint32_t kSmem = kCtas == 2 || kMisc + 1024 > 116 * 1024 ? kMisc + 1024 : 116 * 1024;
  static_assert(kSmem <= 232448 && kCtas * (kSmem + 1024) <= 233472, "shared memory of an SM's CTAs");
  static_assert(kTiles * D <= kSCol && 2 * kTiles * kKeys <= kTmemCols - kSCol, "tensor memory");
};

// What a CTA works on at a time: kTiles tiles of query rows of a sequence and
// key head.  A unit is a token (of a group of more than 128 heads, a token and
// 128 of its heads); a tile holds tile_tokens of them.
struct Item {
  int32_t token0;              // the sequence's first token
  int32_t n;                   // its tokens; 0: no more items
  int32_t unit0;               // first unit of the block
  int32_t head;                // key head
  int32_t first;               // position of its first token (negative: padding)
  int32_t len;                 // its keys
  int32_t key0;                // row of K and V of its first key
  int32_t shift;               // the rows of keys past the sinks are this much further on
};

// The keys that some token in [t0, t1] of the item's sequence sees.
template <int kKeys>
__device__ __forceinline__ Keys<kKeys> item_keys(const PromptAttentionArgs& a, const Item& it, int32_t t0, int32_t t1) {
  Keys<kKeys> k;
  k.hi = max(0, min(it.len, it.first + t1 + 1));
  k.lo = min(k.hi, first_seen(it.first + t0, a.window));
  k.sinks = min(a.num_sinks, k.lo);
  k.sink_steps = (k.sinks + kKeys - 1) / kKeys;
  k.steps = k.sink_steps + (k.hi - k.lo + kKeys - 1) / kKeys;
  return k;
}

// Which place the lane's request has among up to 32 of them, longest first.
__device__ __forceinline__ uint32_t request_rank(const PromptAttentionArgs& a, int lane) {
  const int32_t len = lane < a.batch_size ? load_global(a.cached.seq_lens + lane) : INT32_MIN;
  uint32_t rank = 0;
  for (int j = 0; j < 32; ++j) {
    const int32_t other = __shfl_sync(kFull, len, j);
    rank += other > len || (other == len && j < lane);
  }
  return rank;
}

// Sequences of the cache: every request has as many block numbers as
// max_seq_len (here of query tokens) takes; up to 32 requests come longest
// first, so that short items are left for the end.
template <int kTiles>
__device__ __forceinline__ Item request_item_at(const PromptAttentionArgs& a, uint32_t index, uint32_t rank, int lane) {
  const uint32_t j = a.kv_heads_div.div(index), block = static_cast<uint32_t>(kTiles * a.tile_tokens);
  const uint32_t per = (static_cast<uint32_t>(a.max_seq_len) * a.chunks + block - 1) / block;
  const uint32_t place = j / per, unit0 = (per - 1 - (j - place * per)) * block;
  Item it{};
  if (place >= static_cast<uint32_t>(a.batch_size)) return it;
  const uint32_t b = a.batch_size > 32 ? place : __ffs(__ballot_sync(kFull, rank == place)) - 1;
  GatherPlan plan;
  if (!gather_plan(a.cached, a.seq_start, a.num_tokens, a.max_seq_len, a.window, a.num_sinks, b, plan)) {
    if (lane == 0 && !a.cached.longer_apart) report(a.status, KVQ_STATUS_BAD_BATCH);
    return it;
  }
  if (unit0 >= static_cast<uint32_t>(plan.n) * a.chunks) return it;
  it.head = static_cast<int32_t>(index - j * a.num_kv_heads);
  it.token0 = plan.token0;
  it.n = plan.n;
  it.unit0 = static_cast<int32_t>(unit0);
  it.first = plan.first;
  it.len = plan.len;
  it.key0 = static_cast<int32_t>(b) * a.cached.rows;
  it.shift = plan.sinks - plan.lo;
  return it;
}

// The block of kTiles tiles with number `index` of all key heads' blocks.
// Sequence b's blocks have the numbers from first(b) = floor(units before it /
// units of a block) + b on: those of the sequences before it are fewer.  The
// last blocks of a sequence, which see the most keys, come first.  One warp
// looks b up.
template <int kTiles>
__device__ __forceinline__ Item item_at(const PromptAttentionArgs& a, uint32_t index, int lane) {
  const uint32_t j = a.kv_heads_div.div(index), block = static_cast<uint32_t>(kTiles * a.tile_tokens);
  Item it{};
  it.head = static_cast<int32_t>(index - j * a.num_kv_heads);
  auto first = [&](int32_t b) {                      // (tokens * chunks stay below 2^31; a bad start is skipped below)
    return static_cast<uint32_t>(load_global(a.seq_start + b)) * static_cast<uint32_t>(a.chunks) / block + b;
  };
  // the largest b < batch_size with first(b) <= j, 32 candidates at a time
  int32_t lo = 0, hi = a.batch_size;                 // first(lo) <= j (or lo = 0), first(hi) > j (or hi = batch_size)
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) / 32, b = lo + step * lane;
    const uint32_t below = __ballot_sync(kFull, b < hi && (lane == 0 || first(b) <= j));
    const int32_t at = 31 - __clz(below);            // (lane 0 always is)
    hi = min(hi, lo + step * (at + 1));
    lo = lo + step * at;
  }
  const int32_t q0 = load_global(a.seq_start + lo), q1 = load_global(a.seq_start + lo + 1);
  const int64_t n = static_cast<int64_t>(q1) - q0;
  if (q0 < 0 || n < 0 || q1 > a.num_tokens || n > a.max_seq_len) {
    if (lane == 0) report(a.status, KVQ_STATUS_BAD_BATCH);
    return it;
  }
  const uint32_t blocks = (static_cast<uint32_t>(n) * a.chunks + block - 1) / block;
  const uint32_t at = j - (static_cast<uint32_t>(q0) * a.chunks / block + lo);     // (wraps where j is before the first)
  if (at >= blocks) return it;
  it.token0 = q0;
  it.n = static_cast<int32_t>(n);
  it.unit0 = static_cast<int32_t>((blocks - 1 - at) * block);
  it.len = it.n;
  it.key0 = q0;
  return it;
}

// kCount (a multiple of 32) columns of scores are asked for; they are there
// after tmem_loaded, which takes the registers through itself so that nothing
// that uses them moves up past the wait.
template <int kCount>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[kCount]) {
#pragma unroll
  for (int i = 0; i < kCount; i += 32) tmem_ld32_start(taddr + i, r + i);
}
template <int kCount>
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[kCount]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < kCount; i += 32) held32(r + i);
}
// kCached: over the e4m3 cache's gathered entries.
template <int D, int kTiles, bool kCached>
__global__ void __launch_bounds__(Shape<D, kTiles>::kThreads, Shape<D, kTiles>::kCtas)
    prompt_attention_kernel(const PromptAttentionArgs a, const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<D, kTiles>;
  constexpr int kKeys = S::kKeys;
  constexpr uint32_t kTmemCols = S::kTmemCols, kSCol = S::kSCol;
  wait_for_previous();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(smem);
  const bool before = smem - smem_raw >= 512;
  const uint32_t bar = before ? smem_u32(smem_raw) : base + S::kMisc;
  const uint32_t k_full = bar, k_empty = k_full + 8 * S::kStages, v_full = k_empty + 8 * S::kStages;     // [kStages]
  const uint32_t v_good = v_full + 8 * S::kStages, v_empty = v_good + 8 * S::kStages;
  // [score buffer]: scores there, weights there, their product done
  const uint32_t s_full = v_empty + 8 * S::kStages, p_full = s_full + 32, o_done = p_full + 32;
  const uint32_t o_free = o_done + 32, drain = o_free + 16;                     // [row tile]
  const uint32_t item_full = drain + 16, item_free = item_full + 8 * kSlots;    // [kSlots]
  const uint32_t q_full = item_free + 8 * kSlots, q_free = q_full + 8, answered = q_free + 8;
  const uint32_t answer = (answered + 8 + 15) & ~15u;                           // of the request for a next item
  uint8_t* words = (before ? smem_raw : smem + S::kMisc) + (answer + 16 - bar);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(words);
  volatile int* s_abort = reinterpret_cast<volatile int*>(words + 4);
  volatile Item* items = reinterpret_cast<volatile Item*>(words + 8);
  static_assert(40 * S::kStages + 3 * 32 + 32 + 16 * kSlots + 24 + 32 + 8 + kSlots * sizeof(Item) <= 512, "barrier layout");

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform for the compiler too
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(s_tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, S::kProductWarps);
      mbar_init(v_full + 8 * i, 1);
      mbar_init(v_good + 8 * i, S::kCheckWarps);
      mbar_init(v_empty + 8 * i, S::kProductWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(o_done + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(o_free + 8 * i, 4);
      mbar_init(drain + 8 * i, 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(item_full + 8 * i, 1);
      mbar_init(item_free + 8 * i, S::kWarps - 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, S::kProductWarps);
    mbar_init(answered, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  allow_dependents();
  const uint32_t tmem = __shfl_sync(kFull, *s_tmem, 0);

  auto have = [&](uint32_t bar, uint32_t phase) {
    const bool ok = warp_wait(bar, phase & 1, s_abort);
    fence_after_sync();
    return ok;
  };
  // Item number k of this CTA (false: none, or given up).
  auto next_item = [&](uint32_t k, Item& it) {
    if (!have(item_full + 8 * (k % kSlots), k / kSlots)) return false;
    const volatile Item& s = items[k % kSlots];
    // (uniform for the compiler too)
    it.token0 = __shfl_sync(kFull, s.token0, 0);
    it.n = __shfl_sync(kFull, s.n, 0);
    it.unit0 = __shfl_sync(kFull, s.unit0, 0);
    it.head = __shfl_sync(kFull, s.head, 0);
    it.first = kCached ? __shfl_sync(kFull, s.first, 0) : 0;
    it.len = __shfl_sync(kFull, s.len, 0);
    it.key0 = __shfl_sync(kFull, s.key0, 0);
    it.shift = kCached ? __shfl_sync(kFull, s.shift, 0) : 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(item_free + 8 * (k % kSlots));
    return it.n > 0;
  };
  // its first and last token
  auto first_token = [&](const Item& it) { return static_cast<int32_t>(a.chunk_div.div(static_cast<uint32_t>(it.unit0))); };
  auto last_token = [&](const Item& it) {
    return min(it.n - 1, static_cast<int32_t>(a.chunk_div.div(static_cast<uint32_t>(it.unit0 + kTiles * a.tile_tokens - 1))));
  };
  auto keys_of_item = [&](const Item& it) { return item_keys<kKeys>(a, it, first_token(it), last_token(it)); };
  // row of K and V of step t's first key
  auto row_of = [&](const Item& it, const Keys<kKeys>& keys, int32_t t) {
    return it.key0 + keys.base(t) + (kCached && t >= keys.sink_steps ? it.shift : 0);
  };
  // The score buffer of a row tile and its key tile `at` (of all items'), and
  // which use of it that is.
  auto buffer_of = [](int tile, uint32_t at) { return 2 * static_cast<uint32_t>(tile) + (at & 1); };
  auto use_of = [](uint32_t at) { return at >> 1; };
  // Steps [full0, full1) of the keys are visible whole to every row with a
  // last key of at least hi and a first (but for the sinks) of at most lo.
  auto full_steps = [&](const Keys<kKeys>& keys, int32_t hi, int32_t lo, int32_t& full0, int32_t& full1) {
    full0 = keys.sink_steps + (max(lo - keys.lo, 0) + kKeys - 1) / kKeys;
    const int32_t whole = min(hi, keys.hi - 1) + 1 - keys.lo;           // positions from keys.lo on
    full1 = keys.sink_steps + (whole > 0 ? whole / kKeys : 0);
  };

  Item it;
  if (warp < S::kSoftmaxWarps) {
    // ---- softmax: thread = query row ----------------------------------------
    if constexpr (S::kSplitRegs) more_registers<S::kSoftmaxRegs>();
    const int tile = warp >> 2;
    const uint32_t lanes = (warp & 3) * 32u << 16;
    const uint32_t o_col = tmem + lanes + tile * D;
    const float sc = a.scale_log2;
    uint32_t tiles = 0;                             // of the items before
    for (uint32_t k = 0; next_item(k, it); ++k) {
      const Keys<kKeys> keys = keys_of_item(it);
      // the thread's row: its token (at most the sequence's last) and head
      const uint32_t row = threadIdx.x & 127, unit = static_cast<uint32_t>(it.unit0 + tile * a.tile_tokens);
      uint32_t token_of = a.group_div.div(row), head_of = row - token_of * a.group;
      bool has_row = token_of < static_cast<uint32_t>(a.tile_tokens);
      token_of += unit;
      if (a.chunks > 1) {
        token_of = a.chunk_div.div(unit);
        head_of = (unit - token_of * a.chunks) * 128 + row;
        has_row = head_of < static_cast<uint32_t>(a.group);
      }
      has_row = has_row && token_of < static_cast<uint32_t>(it.n);
      const int32_t token_in = min(static_cast<int32_t>(token_of), it.n - 1);
      const int32_t pos = it.first + token_in, pos_hi = min(pos, it.len - 1);
      const int32_t q_head = it.head * a.group + static_cast<int32_t>(head_of);
      const int32_t pos_lo = first_seen(pos, a.window);
      int32_t full0, full1;
      full_steps(keys, __reduce_min_sync(kFull, pos_hi), __reduce_max_sync(kFull, pos_lo), full0, full1);

      float m = -INFINITY, l = 0.0f;                // reference maximum, sum
      bool done = true;                             // every wait was met
      // which of a step's keys exist, asked for a step ahead
      uint32_t there[3] = {kFull, kFull, kFull};
      auto ask_there = [&](int32_t t) {
        if (kCached && t < keys.steps) {
          const uint32_t* words = a.cached.there + (row_of(it, keys, t) >> 5);
#pragma unroll
          for (int c = 0; c < 3; ++c) there[c] = load_global(words + c);
        }
      };
      ask_there(0);
      for (int32_t t = 0; t < keys.steps; ++t) {
        const uint32_t at = tiles + t, buf = buffer_of(tile, at), use = use_of(at);
        const uint32_t s_col = tmem + lanes + kSCol + kKeys * buf;
        if (!have(s_full + 8 * buf, use)) {
          done = false;
          break;
        }
        uint32_t see[2] = {kFull, kFull};
        if constexpr (kCached) {
          const uint32_t by = row_of(it, keys, t) & 31;
          see[0] = __shfl_sync(kFull, __funnelshift_r(there[0], there[1], by), 0);
          see[1] = __shfl_sync(kFull, __funnelshift_r(there[1], there[2], by), 0);
          ask_there(t + 1);
        }
        const bool masked = t < full0 || t >= full1 || (kCached && (see[0] & see[1]) != kFull);
        if (masked) {
          const int32_t p0 = keys.base(t), end = min(pos_hi, keys.limit(t) - 1);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            see[c] &= range_bits(p0 + 32 * c, pos_lo, end) | range_bits(p0 + 32 * c, 0, min(a.num_sinks - 1, end));
        }
        uint32_t s[kKeys], p[kKeys / 2];
        float sum;
        auto pass = [&](auto with_mask) {           // weights against the reference m: p and their sum
          const float off = m == -INFINITY ? 0.0f : -m;
          float2 sums[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int i = 0; i < kKeys; i += 2) {
            float2 z = ffma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), make_float2(sc, sc),
                             make_float2(off, off));
            if constexpr (with_mask.value) {
              z.x = (see[i >> 5] >> (i & 31)) & 1 ? z.x : -INFINITY;
              z.y = (see[i >> 5] >> ((i + 1) & 31)) & 1 ? z.y : -INFINITY;
            }
            const float2 w = make_float2(ex2(z.x), ex2(z.y));
            sums[(i >> 1) & 1] = fadd2(sums[(i >> 1) & 1], w);
            p[i >> 1] = pack_bf16x2(w.x, w.y);
          }
          const float2 both = fadd2(sums[0], sums[1]);
          sum = both.x + both.y;
        };
        auto weights = [&]() {                      // warp-uniform choice
          if (masked)
            pass(std::true_type{});
          else
            pass(std::false_type{});
        };
        tmem_load(s_col, s);
        tmem_loaded(s);
        // (a row takes a new reference of its own accord, so that its bits do not
        // depend on its neighbours'; the queries of rows that are none may be anything)
        bool behind = has_row;
        if (t > 0) {
          weights();
          behind = has_row && (m == -INFINITY || !(sum <= kMaxSum));
        }
        if (__any_sync(kFull, behind)) {
          if (t > 0) {
            tmem_load(s_col, s);
            tmem_loaded(s);
          }
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < kKeys; ++i) {
            const float z = __uint_as_float(s[i]) * sc;
            if (!masked || ((see[i >> 5] >> (i & 31)) & 1)) top = fmaxf(top, z);
          }
          float alpha = 1.0f;
          if (behind && top > m) {
            alpha = ex2(m - top);                   // 0 while m is -inf
            m = top;
          }
          weights();
          l *= alpha;
          if (t > 0) {
            // O is rescaled once the product of the tile before is done
            if (!have(o_done + 8 * (buf ^ 1), use_of(at - 1))) {
              done = false;
              break;
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tmem_ld32(o_col + 32 * c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
              tmem_st32(o_col + 32 * c, o);
            }
          }
        }
        l += sum;
        tmem_st32_start(s_col, p);
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * buf);
      }
      // the last product is done: O is complete
      tiles += keys.steps;
      if (done && keys.steps > 0) done = have(o_done + 8 * buffer_of(tile, tiles - 1), use_of(tiles - 1));
      if (!done) break;                             // uniform over the warp
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      // The rows leave in pieces of 64 values (128 bytes), eight lanes to a
      // piece, through the warp's 4 KB of shared memory.
      const uint32_t stage = base + S::kOut + warp * 4096;
      const int64_t token = static_cast<int64_t>(it.token0) + token_in;
      const uint64_t mine =
          has_row ? reinterpret_cast<uint64_t>(static_cast<__nv_bfloat16*>(a.out) + token * a.out_stride_t +
                                               q_head * a.out_stride_h)
                  : 0;
      uint64_t to[8];                               // of rows 4 i + lane / 8
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int from = 4 * i + (lane >> 3);
        to[i] = static_cast<uint64_t>(__shfl_sync(kFull, static_cast<uint32_t>(mine >> 32), from)) << 32 |
                __shfl_sync(kFull, static_cast<uint32_t>(mine), from);
      }
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float o[32];
          if (!kCached || keys.steps > 0) {
            tmem_ld32(o_col + 64 * c + 32 * half, o);
          } else {                                  // rows that see nothing
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= inv;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared16(stage + sw128_offset(lane, 4 * half + j),
                        make_uint4(pack_bf16x2(o[8 * j], o[8 * j + 1]), pack_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                   pack_bf16x2(o[8 * j + 4], o[8 * j + 5]), pack_bf16x2(o[8 * j + 6], o[8 * j + 7])));
        }
        if (c == D / 64 - 1 && (!kCached || keys.steps > 0)) {
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free + 8 * tile);
        }
        __syncwarp();
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = ld_shared16(stage + sw128_offset(4 * i + (lane >> 3), lane & 7));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (to[i] != 0) st16(reinterpret_cast<uint8_t*>(to[i]) + 128 * c + 16 * (lane & 7), v[i]);
        __syncwarp();                               // read before the next piece, whose load is the whole warp's
      }
      if (has_row && a.lse != nullptr)
        a.lse[token * a.lse_stride_t + q_head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  } else {
    if constexpr (S::kSplitRegs) fewer_registers<S::kOtherRegs>();
    const uint32_t elected = elect_lane();
    if (warp == S::kCopyWarp) {
      // ---- items, and the copies of K and V ------------------------------------
      uint32_t tiles = 0;                           // of the items before
      uint32_t copied[2] = {0, 0};                  // tiles of K, of V
      uint32_t asked = 0;                           // requests for a next item
      bool waiting = false;                         // one is under way
      uint32_t queries = 0;                         // items whose queries were asked for
      const uint32_t rank = kCached && a.batch_size <= 32 ? request_rank(a, lane) : 0;
      auto block_item = [&](uint32_t index) {
        if constexpr (kCached) return request_item_at<kTiles>(a, index, rank, lane);
        return item_at<kTiles>(a, index, lane);
      };
      it = block_item(blockIdx.x);
      for (uint32_t k = 0;; ++k) {
        // an empty item is passed over; the request for the next one is under way
        // while the keys of this one are copied
        bool ok = true, more = true;
        auto ask = [&]() {
          if (elected) {
            mbar_arrive_expect_tx(answered, 16);
            ask_for_cta(answer, answered);
          }
          __syncwarp();
          waiting = true;
        };
        auto take = [&]() {
          ok = have(answered, asked);
          if (!ok) return;
          waiting = false;
          ++asked;
          const int64_t x = cta_of(answer);
          fence_async_smem();                       // read before the next answer
          __syncwarp();
          more = x >= 0;
          it = Item{};
          if (more) it = block_item(static_cast<uint32_t>(x));
        };
        if (k > 0) take();
        while (ok && more && it.n == 0) {
          ask();
          take();
        }
        if (!ok || (k >= kSlots && !have(item_free + 8 * (k % kSlots), k / kSlots - 1))) break;
        if (lane == 0) {
          volatile Item& s = items[k % kSlots];
          s.token0 = it.token0;
          s.n = it.n;
          s.unit0 = it.unit0;
          s.head = it.head;
          s.first = it.first;
          s.len = it.len;
          s.key0 = it.key0;
          s.shift = it.shift;
          mbar_arrive(item_full + 8 * (k % kSlots));
        }
        __syncwarp();
        if (it.n == 0) break;
        ask();
        const Keys<kKeys> keys = keys_of_item(it);
        if (kCached && keys.steps == 0) continue;
        // the query rows: the tile's tokens and heads as a box (heads past the
        // group's and tokens past the sequence's are rows that no one stores)
        if (queries > 0 && !have(q_free, queries - 1)) break;
        if (elected) {
          mbar_arrive_expect_tx(q_full, kTiles * S::kBlocks * 128 * a.tile_tokens * min(a.group, 128));
#pragma unroll
          for (int w = 0; w < kTiles; ++w) {
            const int32_t unit = it.unit0 + w * a.tile_tokens;
            const int32_t token = a.chunks > 1 ? static_cast<int32_t>(a.chunk_div.div(static_cast<uint32_t>(unit))) : unit;
#pragma unroll
            for (int i = 0; i < S::kBlocks; ++i)
              tma_load_3d(base + w * S::kQTile + i * S::kQBlock, &qmap, 64 * i,
                          it.head * a.group + (unit - token * a.chunks) * 128, it.token0 + token, q_full);
          }
        }
        __syncwarp();
        ++queries;
        auto copy = [&](int32_t t, uint32_t full, uint32_t empty, uint32_t to, const CUtensorMap* map, uint32_t& count) {
          const uint32_t at = tiles + t, st = at % S::kStages;
          if (at >= S::kStages && !have(empty + 8 * st, at / S::kStages - 1)) return false;
          const int32_t key = row_of(it, keys, t);
          if (elected) {
            mbar_arrive_expect_tx(full + 8 * st, S::kTileBytes);
#pragma unroll
            for (int i = 0; i < S::kBlocks; ++i)
              tma_load_3d(base + to + st * S::kTileBytes + i * S::kKBlock, map, 64 * i, it.head, key, full + 8 * st);
          }
          __syncwarp();
          ++count;
          return true;
        };
        auto copy_k = [&](int32_t t) { return t >= keys.steps || copy(t, k_full, k_empty, S::kK, &kmap, copied[0]); };
        if (S::kKeysFirst == 1) ok = copy_k(0);
        for (int32_t t = 0; t < keys.steps && ok; ++t)
          ok = copy_k(t + S::kKeysFirst) && copy(t, v_full, v_empty, S::kV, &vmap, copied[1]);
        if (!ok) break;
        tiles += keys.steps;
      }
      // no copy or answer outlives the CTA (bounded, whatever the abort flag says)
      const long long start = clock64();
      if (waiting)
        while (!mbar_try_wait(answered, asked & 1))
          if (clock64() - start > kDrainCycles) break;
      if (queries > 0)
        while (!mbar_try_wait(q_full, (queries - 1) & 1))
          if (clock64() - start > kDrainCycles) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        for (uint32_t i = copied[x] > S::kStages ? copied[x] - S::kStages : 0; i < copied[x]; ++i)
          while (!mbar_try_wait((x == 0 ? k_full : v_full) + 8 * (i % S::kStages), (i / S::kStages) & 1))
            if (clock64() - start > kDrainCycles) break;
      }
      __syncwarp();
    } else if (warp < S::kCheckWarp) {
      // ---- a row tile's products (one elected lane; the warp waits together) ---
      const int w = warp - S::kProductWarp;
      constexpr uint32_t kIdescS = idesc_bf16(128, kKeys, false), kIdescO = idesc_bf16(128, D, true);
      const uint64_t qdesc = sw128_desc(base + w * S::kQTile, 16, 1024), kdesc = sw128_desc(base + S::kK, 16, 1024);
      const uint64_t vdesc = sw128_desc(base + S::kV, S::kKBlock, 1024);
      const uint32_t o = tmem + w * D;
      uint32_t tiles = 0, items_done = 0;           // of the items before, those items that have any
      bool ok = true;
      for (uint32_t k = 0; ok && next_item(k, it); ++k) {
        const int32_t n = keys_of_item(it).steps;
        if (kCached && n == 0) continue;
        auto keys_there = [&](int32_t t) { return have(k_full + 8 * ((tiles + t) % S::kStages), (tiles + t) / S::kStages); };
        // S(t) = Q K(t)^T
        auto scores = [&](int32_t t) {
          const uint32_t st = (tiles + t) % S::kStages, buf = buffer_of(w, tiles + t);
          const uint64_t kd = kdesc + ((st * S::kTileBytes) >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            warp_mma(elected, tmem + kSCol + kKeys * buf, qdesc + (((ks >> 2) * S::kQBlock + 32 * (ks & 3)) >> 4),
                     kd + (((ks >> 2) * S::kKBlock + 32 * (ks & 3)) >> 4), kIdescS, ks != 0);
          warp_commit(elected, s_full + 8 * buf);
          warp_commit(elected, k_empty + 8 * st);
          if (t == n - 1) warp_commit(elected, q_free);
        };
        ok = have(q_full, items_done);
        for (int32_t t = 0; t < min(n, S::kAhead) && ok; ++t) {
          ok = keys_there(t);
          if (ok) scores(t);
        }
        if (ok && items_done > 0) ok = have(o_free + 8 * w, items_done - 1);
        for (int32_t t = 0; t < n && ok; ++t) {
          const uint32_t st = (tiles + t) % S::kStages, buf = buffer_of(w, tiles + t), use = use_of(tiles + t);
#ifdef KVQ_ATTN_STALL_TILE
          // Failure-detection build only: no product from this tile on, as if
          // the tensor work never completed; the other roles' bounded waits run out.
          if (t == KVQ_ATTN_STALL_TILE) {
            ok = false;
            break;
          }
#endif
          // O += P(t) V(t)
          ok = have(v_good + 8 * st, (tiles + t) / S::kStages);
          if (!S::kKeysLast && ok && t + S::kAhead < n) ok = keys_there(t + S::kAhead);
          const uint64_t vd = vdesc + ((st * S::kTileBytes) >> 4);
          auto product = [&](int ks) {
            warp_mma_ta(elected, o, tmem + kSCol + kKeys * buf + 8 * ks, vd + ((2048 * ks) >> 4), kIdescO,
                        (t > 0 || ks > 0) ? 1u : 0u);
          };
          if (!ok || !(ok = have(p_full + 8 * buf, use))) break;
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks) product(ks);
          warp_commit(elected, o_done + 8 * buf);
          warp_commit(elected, v_empty + 8 * st);
          if (t + S::kAhead < n) {
            if (S::kKeysLast) ok = keys_there(t + S::kAhead);
            if (ok) scores(t + S::kAhead);
          }
        }
        tiles += n;
        ++items_done;
      }
      // the products still in flight are drained (bounded, whatever the abort flag says)
      warp_commit(elected, drain + 8 * w);
      const long long start = clock64();
      while (!mbar_try_wait(drain + 8 * w, 0)) {
        if (clock64() - start > kDrainCycles) {
          *s_abort = 1;
          break;
        }
      }
      __syncwarp();
    } else {
      // ---- V where some row does not see the whole tile ------------------------
      const int me = warp - S::kCheckWarp;
      if (!kCached && blockIdx.x == 0 && me == 0) {   // sequences that item_at may not come across
        for (int32_t b = lane; b < a.batch_size; b += 32) {
          const int32_t q0 = load_global(a.seq_start + b), q1 = load_global(a.seq_start + b + 1);
          if (q0 < 0 || q1 < q0 || q1 > a.num_tokens || static_cast<int64_t>(q1) - q0 > a.max_seq_len)
            report(a.status, KVQ_STATUS_BAD_BATCH);
        }
      }
      uint32_t tiles = 0;
      bool ok = true;
      for (uint32_t k = 0; ok && next_item(k, it); ++k) {
        const Keys<kKeys> keys = keys_of_item(it);
        const int32_t hi = min(it.len - 1, it.first + first_token(it));
        const int32_t lo = first_seen(it.first + last_token(it), a.window);
        int32_t full0, full1;
        full_steps(keys, hi, lo, full0, full1);
        for (int32_t t = 0; t < keys.steps; ++t) {
          const uint32_t at = tiles + t, st = at % S::kStages;
          ok = have(v_full + 8 * st, at / S::kStages);
          if (!ok) break;
          if (t < full0 || t >= full1) {
            // Rows of the tile: those from `there` on are no keys (zeros); of the
            // others, [all0, all1) are visible to every query and stay as they are.
            const int32_t there = keys.limit(t) - keys.base(t);
            const int32_t all0 = t < keys.sink_steps ? 0 : max(0, lo - keys.base(t));
            const int32_t all1 = min(there, hi + 1 - keys.base(t));
            uint4* v = reinterpret_cast<uint4*>(smem + S::kV + st * S::kTileBytes) + lane;
            constexpr int kRows = 4, kBatch = 8;                  // rows to a load of the warp; loads under way at once
#pragma unroll 1
            for (int32_t r = kRows * kBatch * me; r < kKeys; r += kRows * kBatch * S::kCheckWarps) {
              if (r >= all0 && r + kRows * kBatch <= all1) continue;
#pragma unroll 1
              for (int block = 0; block < S::kBlocks; ++block) {
                uint4* row = v + block * (S::kKBlock / 16) + r * 8;
                uint4 x[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) x[j] = row[32 * j];
                constexpr uint32_t kAbs = 0x7FFF7FFFu;
                uint32_t top = 0;                                 // largest bits below the signs, of either half
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                  top = __vimax3_u16x2(top, x[j].x & kAbs, x[j].y & kAbs);
                  top = __vimax3_u16x2(top, x[j].z & kAbs, x[j].w & kAbs);
                }
                if (r + kRows * kBatch > there || (top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u) {
                  auto finite = [](uint32_t w) {
                    return ((w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
                  };
#pragma unroll
                  for (int j = 0; j < kBatch; ++j) {
                    const int32_t at = r + kRows * j + lane / 8;
                    if (at >= all0 && at < all1) continue;
                    row[32 * j] = at < there ? make_uint4(finite(x[j].x), finite(x[j].y), finite(x[j].z), finite(x[j].w))
                                             : make_uint4(0, 0, 0, 0);
                  }
                }
              }
            }
            fence_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(v_good + 8 * st);
        }
        tiles += keys.steps;
      }
    }
  }

  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *s_abort) report(a.status, KVQ_STATUS_TIMEOUT);
  if (warp == 0) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(*s_tmem), "r"(kTmemCols) : "memory");
  }
}

// Tensor map of the queries [tokens][heads][D], tiles of 64 dimensions of a
// group's heads of tile_tokens tokens with the 128-byte swizzle.
bool query_tensor_map(const PromptAttentionArgs& a, CUtensorMap* map) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.head_size), static_cast<cuuint64_t>(a.num_heads),
                              static_cast<cuuint64_t>(a.num_tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.q_stride_h) * 2, static_cast<cuuint64_t>(a.q_stride_t) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.group < 128 ? a.group : 128),
                             static_cast<cuuint32_t>(a.tile_tokens)};
  const cuuint32_t elem_strides[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, elem_strides,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of keys or values [tokens][heads][D], tiles of 64 dimensions of
// kKeys tokens of one head with the 128-byte swizzle; tokens past the last
// one are zero-filled.
template <int D, int kKeys>
bool key_tensor_map(const void* p, int64_t stride_t, int64_t stride_h, int32_t heads, int64_t tokens, CUtensorMap* map) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride_h) * 2, static_cast<cuuint64_t>(stride_t) * 2};
  const cuuint32_t box[3] = {64, 1, kKeys}, elem_strides[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, elem_strides,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int kTiles, bool kCached>
cudaError_t launch(const PromptAttentionArgs& a, cudaStream_t stream) {
  using S = Shape<D, kTiles>;
  const int64_t rows = kCached ? int64_t{a.cached.rows} * a.batch_size : a.num_tokens;
  CUtensorMap qmap, kmap, vmap;
  if (!query_tensor_map(a, &qmap) || !key_tensor_map<D, S::kKeys>(a.k, a.k_stride_t, a.k_stride_h, a.num_kv_heads, rows, &kmap) ||
      !key_tensor_map<D, S::kKeys>(a.v, a.v_stride_t, a.v_stride_h, a.num_kv_heads, rows, &vmap))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(prompt_attention_kernel<D, kTiles, kCached>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t block = kTiles * a.tile_tokens;
  const int64_t blocks = kCached ? (int64_t{a.max_seq_len} * a.chunks + block - 1) / block * a.batch_size
                                 : a.num_tokens * a.chunks / block + a.batch_size;          // the numbers of item_at
  return launch_dependent(prompt_attention_kernel<D, kTiles, kCached>, dim3(static_cast<unsigned>(blocks * a.num_kv_heads)),
                          S::kThreads, S::kSmem, 1, stream, a, qmap, kmap, vmap);
}

template <bool kCached>
cudaError_t launch_size(const PromptAttentionArgs& a, cudaStream_t stream) {
  // two row tiles share a key tile wherever a sequence can fill them
  const bool two = static_cast<int64_t>(a.max_seq_len) * a.chunks > a.tile_tokens;
  switch (a.head_size) {
    case 64: return two ? launch<64, 2, kCached>(a, stream) : launch<64, 1, kCached>(a, stream);
    case 128: return two ? launch<128, 2, kCached>(a, stream) : launch<128, 1, kCached>(a, stream);
    default: return launch<256, 1, kCached>(a, stream);   // one tile's O fills half of the tensor memory
  }
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptAttentionArgs& a, cudaStream_t stream) {
  return a.cached.there != nullptr ? launch_size<true>(a, stream) : launch_size<false>(a, stream);
}

}  // namespace kvq
