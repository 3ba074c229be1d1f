// kvq_per_head_prefill.cu -- the attention over the paged per-head NVFP4
// cache (window and tree masks, defined in kvq_per_head_attention.cu) for
// many query rows that share a key head: chunks of new tokens, large draft
// trees.  The products bound it: 4 D flops for each (row, visible key).
//
// Design: one CTA per (block of 128 kTiles query rows, key head, range of
// keys), one CTA per SM; the rows are (token, head) pairs of one request.
// Two row tiles (kTiles = 2) share every decoded tile of 64 keys, and their
// softmax and products alternate.
//   - tensor memory: O of row tile w in columns [D w, +D); its scores S (128 x
//     64 fp32) in two buffers from column 256 on, so that the scores of tile t
//     + 1 are formed while the weights of tile t are computed; the weights P
//     (f16) overwrite the first half of their S.  (128 keys per tile would
//     leave room for one buffer: product, scores and weights of a row tile
//     then wait for one another, 5900 clocks per 128 keys where the products
//     need 2048.)
//   - shared memory: q in f16 (scaled by each row's power of two), K tiles and
//     V tiles (64 x D f16, 128-byte swizzle, kStages of each), and a ring of
//     raw entries per side;
//   - some warps decode the keys and as many the values: raw entries come in by
//     asynchronous copies, kRing chunks ahead (each warp copies what it
//     decodes, so that it waits for no other); 8 lanes take 8 rows of a
//     64-column block, so that their 16-byte stores fall in different banks;
//   - one warp issues the scores' products S_w(t) = Q_w K(t)^T, another the
//     outputs' O_w += P_w(t) V(t): a wait costs either about 200 clocks, which
//     the other's products cover;
//   - four softmax warps per row tile, one thread per row, in one pass over
//     the scores: the weights are formed against the reference maximum of the
//     tiles before, without a maximum of their own; only when their sum shows
//     that one of them may exceed it by 2^8 is the tile's maximum taken, the
//     pass repeated and O rescaled.
// Measured: 4 requests x 4096 new tokens x 32 heads (8 key heads) of 128,
// window 4096: 860 us = 1279 TFLOP/s, about 1700 clocks per pair of row tiles
// and 64 keys, of which the products take 1280 (768 for the scores, whose 64
// columns run at two thirds of the full rate).  The softmax warps set the pace: about
// 1000 clocks for the exponentials, sums and f16 weights of the two row tiles
// on an SM quarter (512 by the exponentials' rate alone, 530 when nothing else
// runs there), the rest for loads, stores and waits.  Making the two row
// tiles take turns at it cost more (1115 us) than the contention (943 then).
// Every wait of a role on another role or on its products is bounded; on
// expiry the CTA records KVQ_STATUS_TIMEOUT, drains its products, frees its
// tensor memory and leaves its rows unwritten.  (The set-up waits otherwise:
// for the kernel before, at the block's barrier, which every thread reaches,
// and for tensor memory, which whoever holds it gives back without this CTA.)
#include <type_traits>

#include "kvq_per_head_attention.cuh"
#include "kvq_per_head_plan.h"

namespace kvq {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;
constexpr int64_t kMaxPos = INT32_MAX - 256;      // positions stay below it (host check)
constexpr int kKeys = 64;                         // keys per tile
constexpr int kValidRing = 16;
constexpr uint32_t kBlockBytes = 128 * 128;       // 64 dimensions of 128 rows of q
constexpr uint32_t kKBlock = kKeys * 128;         // 64 dimensions of a key tile

template <int D, int kTiles>
struct Shape {
  // Warps: softmax; those that decode keys, and the one that issues the
  // scores' products; those that decode values, and the one that issues the
  // outputs'; in whole warpgroups, whose registers are split by role (the
  // threads start with an equal share, and the shares add up to no more).
  static constexpr int kSoftmaxWarps = 4 * kTiles;
  static constexpr int kKeyWarps = kTiles == 2 ? 3 : 5, kValueWarps = kKeyWarps;
  static constexpr int kScoreWarp = kSoftmaxWarps + kKeyWarps;
  static constexpr int kOutputWarp = kScoreWarp + 1 + kValueWarps;
  static constexpr int kThreads = 32 * (kOutputWarp + 1);
  static_assert(kThreads == 512, "warpgroups");
  static constexpr int kStartRegs = 128;
  // (two row tiles: 152 / 104 and 136 / 120 spill in the loops; 4 x 4096 tokens
  // 898 us with the former, 861 with 144 / 112)
  static constexpr int kSoftmaxRegs = kTiles == 2 ? 144 : 200;
  static constexpr int kOtherRegs = kTiles == 2 ? 112 : 96;
  static_assert(32 * kSoftmaxWarps * kSoftmaxRegs + (kThreads - 32 * kSoftmaxWarps) * kOtherRegs <=
                    kThreads * kStartRegs, "register split");
  static constexpr int kBlocks = D / 64;                     // 64-dimension blocks
  static constexpr int kStages = D == 256 ? 2 : 3;           // decoded tiles of K, of V
  static constexpr uint32_t kTileBytes = kBlocks * kKBlock;
  static constexpr uint32_t kQTile = kBlocks * kBlockBytes;
  static constexpr uint32_t kK = kTiles * kQTile;
  static constexpr uint32_t kV = kK + kStages * kTileBytes;
  // raw entries of one side: rings of chunks of keys, data rows then scale rows
  static constexpr int kChunk = D == 256 ? 32 : 64;
  static constexpr int kParts = kKeys / kChunk;              // chunks per tile
  static constexpr int kRing = D == 256 ? 3 : 4;
  static constexpr uint32_t kRawScales = kChunk * (D / 2);
  static constexpr uint32_t kRawBytes = kRawScales + kChunk * (D / 16);
  static constexpr uint32_t kRawK = kV + kStages * kTileBytes;
  static constexpr uint32_t kRawV = kRawK + kRing * kRawBytes;
  static constexpr uint32_t kMisc = kRawV + kRing * kRawBytes;
  // at least 116 KB, so that a second CTA, which would wait for tensor memory, does not share the SM
  static constexpr uint32_t kSmem = kMisc + 512 + 1024 > 116 * 1024 ? kMisc + 512 + 1024 : 116 * 1024;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(kTiles * D <= 256 && kMisc % 16 == 0, "tensor memory, alignment");
};

// warp_wait_or_abort whose usual case, the phase complete already, takes one
// test, without the clock, the loop and the suspension of a waiting try
// (trees 32 x 64: 576 -> 566 us).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* s_abort) {
  return __all_sync(kFull, mbar_test_wait(bar, parity)) || warp_wait_or_abort(bar, parity, s_abort);
}

// The CTA's set-up is done (tensor memory, barriers): every role comes here
// once, after what it can start before.
__device__ __forceinline__ void set_up_done() {
  fence_before_sync();
  asm volatile("bar.sync 0;" ::: "memory");
  fence_after_sync();
}

// kind::f16 with f16 operands, fp32 sums; A is K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// Bits i (0..31) with lo <= p0 + i <= hi.
__device__ __forceinline__ uint32_t range_bits(int32_t p0, int32_t lo, int32_t hi) {
  const int32_t a = max(lo - p0, 0), b = min(hi - p0, 31);
  return a > b ? 0u : (0xffffffffu >> (31 - b)) & (0xffffffffu << a);
}

// Bits d .. d + 31 of a mask row (bits outside it are 0).
__device__ __forceinline__ uint32_t tree_bits(const uint64_t* row, int32_t words, int64_t d) {
  if (d <= -32) return 0;
  if (d < 0) return static_cast<uint32_t>(load_global(row) << static_cast<int>(-d));
  const int64_t w = d >> 6;
  const int sh = static_cast<int>(d & 63);
  uint64_t v = w < words ? load_global(row + w) >> sh : 0;
  if (sh > 32 && w + 1 < words) v |= load_global(row + w + 1) << (64 - sh);
  return static_cast<uint32_t>(v);
}

// A producer lane's piece of one entry side: D / 4 codes and their scales.
template <int D>
struct Piece {
  static constexpr int kWords = D / 32;              // 32-bit words of codes (8 codes each)
  uint32_t w[kWords];
  uint32_t sf;
};

// Byte offset of part i of lane part k (0..3) of raw row r: rows are D / 2
// bytes apart, their pieces permuted so that 8 rows' reads of one part fall
// in different banks.  (The permutation repeats every 8 rows.)
template <int D>
__device__ __forceinline__ uint32_t raw_offset(uint32_t r, uint32_t k, uint32_t i) {
  if constexpr (D == 64) return r * 32 + 8 * (k ^ ((r >> 1) & 2));
  if constexpr (D == 128) return r * 64 + 16 * (k ^ ((r >> 1) & 3));
  return r * 128 + 16 * ((2 * k + i) ^ (r & 7));
}

// A lane's places in the raw ring and in the decoded tiles, for the row of
// its first pass; a later pass's are a whole number of 8-row groups on.
template <int D>
struct Lane {
  uint32_t raw[D == 256 ? 2 : 1], sf, tile[D / 32];
  __device__ __forceinline__ Lane(uint32_t r, uint32_t k, uint32_t scales) {
#pragma unroll
    for (int i = 0; i < (D == 256 ? 2 : 1); ++i) raw[i] = raw_offset<D>(r, k, i);
    sf = scales + r * (D / 16) + (D / 64) * k;
    // D / 4 dimensions: block (D / 4) k / 64, chunks from ((D / 4) k % 64) / 8 on
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      tile[j] = (D * k / 256) * kKBlock + r * 128u + ((((D / 32 * k) & 7) + j) ^ (r & 7u)) * 16u;
  }
};

template <int D>
__device__ __forceinline__ void load_piece(uint32_t raw, const Lane<D>& at, int groups, Piece<D>& e) {
  if constexpr (D == 64) {
    const uint2 v = lds64(raw + at.raw[0] + groups * 8 * (D / 2));
    e.w[0] = v.x;
    e.w[1] = v.y;
    e.sf = lds8(raw + at.sf + groups * 8 * (D / 16));
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const uint4 v = ld_shared16(raw + at.raw[i] + groups * 8 * (D / 2));
      e.w[4 * i] = v.x;
      e.w[4 * i + 1] = v.y;
      e.w[4 * i + 2] = v.z;
      e.w[4 * i + 3] = v.w;
    }
    const uint32_t sf = raw + at.sf + groups * 8 * (D / 16);
    e.sf = D == 128 ? lds16(sf) : lds32(sf);
  }
}

// Decodes a piece and stores its 16-byte chunks into its row of a tile.
template <int D, bool kValues>
__device__ __forceinline__ void store_piece(uint32_t tile, const Lane<D>& at, int groups, const Piece<D>& e) {
#pragma unroll
  for (int p = 0; p < (D + 127) / 128; ++p) {        // two scales at a time
    uint32_t s2 = bits(e4m3x2_to_half2(e.sf >> (16 * p)));
    if constexpr (kValues) s2 = finite_scales(s2);
#pragma unroll
    for (int j = 0; j < (D == 64 ? 2 : 4); ++j) {
      const uint32_t sf = j < 2 ? low_both(s2) : high_both(s2);
      uint32_t h[4];
      e2m1x8(e.w[4 * p + j], h);
      st_shared16(tile + at.tile[4 * p + j] + groups * 1024,
                  make_uint4(hmul2(h[0], sf), hmul2(h[1], sf), hmul2(h[2], sf), hmul2(h[3], sf)));
    }
  }
}

// ---------------------------------------------------------------------------
// producers: the keys or the values of every tile
// ---------------------------------------------------------------------------
//
// kWarps warps share a chunk's rows in groups of 8: warp `me` takes groups me,
// me + kWarps, ... in passes.  Lane l looks up row l of the warp's rows (pass
// l / 8, row l % 8 of its group): page id, loaded a chunk before its copies
// start and looked at only there, address, scale copy.  For the data of pass
// i it is lane part k = l / 8 (dimensions k D / 4 .. +D / 4) of row l % 8.
template <int D, int kTiles, bool kValues>
__device__ __forceinline__ void produce(const PerHeadAttentionArgs& a, int b, uint32_t head, const Keys<kKeys>& keys,
                                        int32_t s0, int32_t n_tiles, int me, int lane, bool bad_index, uint32_t base,
                                        uint32_t full, uint32_t empty, uint8_t* valid_ring,
                                        volatile int* s_abort) {
  using S = Shape<D, kTiles>;
  constexpr int kWarps = kValues ? S::kValueWarps : S::kKeyWarps;
  constexpr int kGroups = S::kChunk / 8, kPasses = (kGroups + kWarps - 1) / kWarps;
  static_assert(kPasses <= 4, "a lane per row");
  const uint32_t k = lane >> 3;
  const uint32_t tiles = base + (kValues ? S::kV : S::kK), raw_ring = base + (kValues ? S::kRawV : S::kRawK);
  const int32_t chunks = n_tiles * S::kParts;
  const uint8_t* side = a.cache + (kValues ? a.region : 0);
  const int32_t* table = a.block_table + b * a.block_table_stride;
  const Lane<D> at(8 * me + (lane & 7), k, S::kRawScales);
  const uint32_t own_row = 8 * (me + kWarps * (lane >> 3)) + (lane & 7);   // of the warp's rows, the one it looks up
  const bool has_row = own_row < S::kChunk && (lane >> 3) < kPasses;
  const uint32_t head_row = head * static_cast<uint32_t>(a.row_head);
  auto look_up = [&](int32_t h) {                   // its position in chunk h
    const int32_t step = s0 + h / S::kParts;
    const uint32_t p = static_cast<uint32_t>(keys.base(step)) + (h % S::kParts) * S::kChunk + own_row;
    return look_up_position(a, table, head_row, has_row && h < chunks && p < static_cast<uint32_t>(keys.limit(step)), p);
  };
  auto start = [&](int32_t h, const LookUp& next) { // one group of copies, empty past the last chunk
    if (h < chunks) {
      const uint32_t raw = raw_ring + (h % S::kRing) * S::kRawBytes;
      const bool ok = next.in && next.id >= 0 && next.id < a.num_pages;
      bad_index = bad_index || (next.in && !ok);
      const uint8_t* region = at_offset(side, ok ? next.id : 0, 2 * a.region);    // some page where there is none
      const uint32_t row = ok ? next.row : 0;
      const uint64_t data = reinterpret_cast<uint64_t>(at_offset(region, row, D / 2));
      if (has_row)
        cp_async<D / 16>(raw + S::kRawScales + own_row * (D / 16), at_offset(region + a.scales, row, D / 16),
                         ok ? D / 16 : 0);
      const uint32_t rows = __ballot_sync(kFull, ok);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int from = 8 * i + (lane & 7);
        const uint64_t row_data =
            static_cast<uint64_t>(__shfl_sync(kFull, static_cast<uint32_t>(data >> 32), from)) << 32 |
            __shfl_sync(kFull, static_cast<uint32_t>(data), from);
        if (me + kWarps * i >= kGroups) continue;   // uniform over the warp
        const bool there = (rows >> from) & 1;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(row_data) + (D / 8) * k;
        constexpr int kPiece = D == 64 ? 8 : 16;
#pragma unroll
        for (int j = 0; j < (D == 256 ? 2 : 1); ++j)
          cp_async<kPiece>(raw + at.raw[j] + i * kWarps * 8 * (D / 2), src + 16 * j, there ? kPiece : 0);
      }
      // Which keys exist, for the softmax.  A slot's last reader is done: with
      // tile t under way here, kRing chunks ahead of it at most, tile t -
      // kStages has left its buffer, so that its scores are formed, for which
      // the weights of tile t - kStages - 2 had to leave theirs.
      static_assert((S::kParts - 1 + S::kRing) / S::kParts + S::kStages + 2 <= kValidRing, "mask slots");
      if constexpr (!kValues) {
        if (lane < kPasses && me + kWarps * lane < kGroups)
          valid_ring[8 * ((h / S::kParts) % kValidRing) + (h % S::kParts) * kGroups + me + kWarps * lane] =
              static_cast<uint8_t>(rows >> (8 * lane));
      }
    }
    cp_commit();
  };
  // The first look-ups are under way before the CTA's set-up is waited for: all
  // of the first chunks', or one (two row tiles: registers).
  LookUp next;
  if constexpr (kTiles == 1) {
    LookUp first[S::kRing];
#pragma unroll
    for (int h = 0; h < S::kRing; ++h) first[h] = look_up(h);
    next = look_up(S::kRing);
    set_up_done();
#pragma unroll
    for (int h = 0; h < S::kRing; ++h) start(h, first[h]);
  } else {
    next = look_up(0);
    set_up_done();
    // (rolled, the code is fetched sooner: short ragged chunks at D = 64 29.3
    // against 31.4 us; at D = 128 it spills in the loop below, 875 against 861)
#pragma unroll (D == 64 ? 1 : S::kRing)
    for (int h = 0; h < S::kRing; ++h) {
      start(h, next);
      next = look_up(h + 1);
    }
  }
  Piece<D> e[kPasses];                              // of the next chunk: read a chunk ahead, all at once
  auto read = [&](int32_t h) {
    cp_wait<S::kRing - 1>();
    __syncwarp();                                   // chunk h is there
    const uint32_t raw = raw_ring + (h % S::kRing) * S::kRawBytes;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (me + kWarps * i < kGroups) load_piece<D>(raw, at, i * kWarps, e[i]);
  };
  read(0);
  for (int32_t h = 0; h < chunks; ++h) {
    const int32_t t = h / S::kParts;
    const int st = t % S::kStages;
    if (h % S::kParts == 0 && t >= S::kStages && !warp_wait(empty + 8 * st, (t / S::kStages - 1) & 1, s_abort)) break;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (me + kWarps * i < kGroups)
        store_piece<D, kValues>(tiles + st * S::kTileBytes + (h % S::kParts) * S::kChunk * 128, at, i * kWarps, e[i]);
    if (h % S::kParts == S::kParts - 1) fence_async_smem();
    __syncwarp();                                   // and chunk h has been read
    if (h % S::kParts == S::kParts - 1 && lane == 0) mbar_arrive(full + 8 * st);
    start(h + S::kRing, next);
    next = look_up(h + S::kRing + 1);
    read(h + 1);
  }
  cp_wait<0>();                                     // no copy outlives the CTA
  if (bad_index && !kValues) report(a.status, KVQ_STATUS_BAD_INDEX);
}

template <int D, int kTiles>
__global__ void __launch_bounds__(Shape<D, kTiles>::kThreads, 1)
    per_head_prefill_kernel(const PerHeadAttentionArgs a, int32_t row_blocks) {
  using S = Shape<D, kTiles>;
  wait_for_previous();
  const float k_scale = load_global(a.k_scale);           // in flight beside the request
  // the last row blocks of a causal chunk, which see the most keys, come first
  const Place place = place_of(a, row_blocks);
  const uint32_t head = place.head;
  const int32_t rb = row_blocks - 1 - place.row_block, split = place.split;
  const int b = blockIdx.y;
  Request rq;
  if (!request_of(a, b, rq)) {                     // uniform over the CTA, as every return up here
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, KVQ_STATUS_BAD_BATCH);
    return;
  }
  const int64_t total_rows = static_cast<int64_t>(rq.tokens) * a.group;
  const int64_t row0 = static_cast<int64_t>(rb) * (128 * kTiles);
  if (row0 >= total_rows) return;
  const int32_t rows = static_cast<int32_t>(min(static_cast<int64_t>(128 * kTiles), total_rows - row0));
  const int32_t t0 = a.group_div.div(static_cast<uint32_t>(row0));
  const int32_t t1 = a.group_div.div(static_cast<uint32_t>(row0 + rows - 1));
  const Keys<kKeys> keys = keys_of<kKeys>(a, rq, t0, t1);
  int32_t s0, s1;
  range_of(a, keys, split, s0, s1);
  if (a.num_splits > 1 && s0 == s1) {
    // an empty range: it weighs nothing when the ranges are joined
    for (int r = threadIdx.x; r < rows; r += S::kThreads) {
      const RowAt at = row_at(a, rq, head, static_cast<uint32_t>(row0 + r));
      a.part_lse[(at.token * a.num_heads + at.head) * a.num_splits + split] = -INFINITY;
    }
    return;
  }
  const int32_t n_tiles = s1 - s0;
  allow_dependents();

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t bar = base + S::kMisc;
  const uint32_t k_full = bar, k_empty = bar + 24, v_full = bar + 48, v_empty = bar + 72;   // [kStages] each
  const uint32_t s_full = bar + 96, p_full = bar + 128, o_done = bar + 160;                 // [row tile][buffer] each
  const uint32_t drain = bar + 192, q_full = bar + 208;            // [2], 1
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + S::kMisc + 216);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + S::kMisc + 220);
  uint8_t* valid_ring = smem + S::kMisc + 224;     // [kValidRing][8]: bit per key of the tile
  static_assert(S::kStages <= 3 && 224 + 8 * kValidRing <= 512, "barrier layout");

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform for the compiler too
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(s_tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(k_full + 8 * i, S::kKeyWarps);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, S::kValueWarps);
      mbar_init(v_empty + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + 8 * i, 2);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(o_done + 8 * i, 1);
    }
    mbar_init(drain, 1);
    mbar_init(drain + 8, 1);
    mbar_init(q_full, S::kSoftmaxWarps);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // Softmax threads: their query row.  Rows past the block's are zero.
  const int32_t row = static_cast<int32_t>(threadIdx.x);
  bool has_row = false;
  int64_t token = 0;
  int32_t q_head = 0, pos_hi = -1, pos_lo = 0;
  uint64_t src = 0;
  auto set_row = [&]() {
    has_row = warp < S::kSoftmaxWarps && row < rows;
    if (!has_row) return;
    const RowAt at = row_at(a, rq, head, static_cast<uint32_t>(row0 + row));
    token = at.token;
    q_head = at.head;
    const int64_t p = rq.first_pos + (token - rq.token0);
    pos_hi = static_cast<int32_t>(max(int64_t{-1}, min(p, static_cast<int64_t>(rq.len) - 1)));
    if (a.window > 0)
      pos_lo = static_cast<int32_t>(min(static_cast<int64_t>(rq.len), max(int64_t{0}, p - a.window + 1)));
    src = reinterpret_cast<uint64_t>(static_cast<const __nv_bfloat16*>(a.q) + token * a.q_stride_t +
                                     q_head * a.q_stride_h);
  };
  if (warp < S::kSoftmaxWarps) {
    // ---- softmax: thread = query row ----------------------------------------
    const int tile = warp >> 2;                     // its row tile
    set_row();
    // The warp's 32 query rows come in as they are, D / 8 lanes to a row,
    // while the CTA sets up; then each thread scales its own in place.  (Short
    // loops: a CTA runs this code once, and fetching it took longer than the
    // loads, 2.1 us with the rows in registers.)
    const uint32_t q_rows = base + tile * S::kQTile + (warp & 3) * (32 * 128);
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
#pragma unroll 4
    for (int i = 0; i < 32; i += kAtOnce) {
      const int from = i + lane / kLanes, c = lane % kLanes;
      const uint64_t at = static_cast<uint64_t>(__shfl_sync(kFull, static_cast<uint32_t>(src >> 32), from)) << 32 |
                          __shfl_sync(kFull, static_cast<uint32_t>(src), from);
      cp_async<16>(q_rows + (c >> 3) * kBlockBytes + sw128_offset(from, c & 7),
                   reinterpret_cast<const uint4*>(at != 0 ? at : reinterpret_cast<uint64_t>(a.q)) + (at != 0 ? c : 0),
                   at != 0 ? 16 : 0);
    }
    cp_commit();
    set_up_done();
    more_registers<S::kSoftmaxRegs>();
    const uint32_t tmem = __shfl_sync(kFull, *s_tmem, 0);
    cp_wait<0>();
    __syncwarp();
    // (eight pieces at a time: the decoding warps' copies keep a load waiting
    // for a hundred clocks)
    uint32_t top = 0;                               // largest bits below the signs, of either half
#pragma unroll 1
    for (int c = 0; c < D / 8; c += 8) {
      const uint32_t at = q_rows + (c >> 3) * kBlockBytes;
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = ld_shared16(at + sw128_offset(lane, i));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        top = __vimax3_u16x2(top, x[i].x & kAbs, x[i].y & kAbs);
        top = __vimax3_u16x2(top, x[i].z & kAbs, x[i].w & kAbs);
      }
    }
    const RowScale rs = row_scale(__uint_as_float(max(top << 16, top & 0xFFFF0000u)));
#pragma unroll 1
    for (int c = 0; c < D / 8; c += 8) {
      const uint32_t at = q_rows + (c >> 3) * kBlockBytes;
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = ld_shared16(at + sw128_offset(lane, i));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = fmul2(fmul2(make_float2(bf16_lo(w[j]), bf16_hi(w[j])), make_float2(rs.f[0], rs.f[0])),
                                 make_float2(rs.f[1], rs.f[1]));
          h[j] = pack_f16x2(v.x, v.y);
        }
        st_shared16(at + sw128_offset(lane, i), make_uint4(h[0], h[1], h[2], h[3]));
      }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    const float sc = a.scale_log2 * k_scale * rs.i[0] * rs.i[1];   // score -> base-2 exponent

    float m = has_row ? -INFINITY : 0.0f, l = 0.0f; // reference maximum, sum
    bool done = true;                               // every wait was met
    const uint32_t lanes = (warp & 3) * 32u << 16;
    const uint32_t o_col = tmem + lanes + tile * D;
    // Steps [full0, full1) of the keys are visible whole to every row of the
    // warp (those whose pages all exist): no mask is looked at there.
    int32_t full0 = keys.sink_steps, full1;
    if (a.tree_mask != nullptr) {
      full1 = rq.first_pos <= 0 ? 0 : static_cast<int32_t>(min(rq.first_pos, static_cast<int64_t>(rq.len)) / kKeys);
    } else {
      const int32_t hi = __reduce_min_sync(kFull, has_row ? pos_hi : INT32_MAX);
      const int32_t lo = __reduce_max_sync(kFull, has_row ? pos_lo : 0);
      full0 += (max(lo - keys.lo, 0) + kKeys - 1) / kKeys;
      const int32_t whole = min(hi, keys.hi - 1) + 1 - keys.lo;        // positions from keys.lo on
      full1 = keys.sink_steps + (whole > 0 ? whole / kKeys : 0);
    }
    bool fresh = true;                              // some row has no reference yet (uniform over the warp)
    for (int32_t t = 0; t < n_tiles; ++t) {
      const int buf = 2 * tile + (t & 1);
      const uint32_t s_col = tmem + lanes + kSCol + kKeys * buf;
      if (!warp_wait(s_full + 8 * buf, (t >> 1) & 1, s_abort)) {
        done = false;
        break;
      }
      fence_after_sync();
      uint32_t s[64], p[32];
      tmem_ld64(s_col, s);

      // which of the tile's keys the row sees
      const uint2 valid = lds64(smem_u32(valid_ring) + 8 * (t % kValidRing));
      const bool masked = s0 + t < full0 || s0 + t >= full1 || (valid.x & valid.y) != kFull;
      uint32_t see[2] = {0, 0};
      if (masked && has_row) {
        const int32_t p0 = keys.base(s0 + t);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int32_t pc = p0 + 32 * c;
          uint32_t w;
          if (a.tree_mask != nullptr)
            w = (rq.first_pos > 0 ? range_bits(pc, 0, static_cast<int32_t>(min(rq.first_pos - 1, kMaxPos))) : 0u) |
                tree_bits(a.tree_mask + token * a.tree_stride, a.tree_words, pc - rq.first_pos);
          else
            w = range_bits(pc, pos_lo, pos_hi) | range_bits(pc, 0, min(a.num_sinks - 1, pos_hi));
          see[c] = (c == 0 ? valid.x : valid.y) & w;
        }
      }
      float sum;
      // weights against the reference m: p and their sum
      auto pass = [&](float off, auto with_mask) {
        float2 sums[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float2 z = ffma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), make_float2(sc, sc),
                           make_float2(off, off));
          if constexpr (with_mask.value) {
            z.x = (see[i >> 5] >> (i & 31)) & 1 ? z.x : -INFINITY;
            z.y = (see[i >> 5] >> ((i + 1) & 31)) & 1 ? z.y : -INFINITY;
          }
          const float2 w = make_float2(ex2(z.x), ex2(z.y));
          sums[(i >> 1) & 1] = fadd2(sums[(i >> 1) & 1], w);
          p[i >> 1] = pack_f16x2(w.x, w.y);
        }
        const float2 both = fadd2(sums[0], sums[1]);
        sum = both.x + both.y;
      };
      auto weights = [&]() {                        // warp-uniform choice
        const float off = kShift - (m == -INFINITY ? 0.0f : m);
        if (masked)
          pass(off, std::true_type{});
        else
          pass(off, std::false_type{});
      };
      // No weight is above 2^(kShift + kGrow) if their sum is not; a row whose
      // sum is takes a new reference, its tile's maximum (as in its first tile).
      if (!fresh) weights();
      if (fresh || __any_sync(kFull, sum > kMaxWeight)) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          const float z = __uint_as_float(s[i]) * sc;
          if (!masked || ((see[i >> 5] >> (i & 31)) & 1)) top = fmaxf(top, z);
        }
        float alpha = 1.0f;
        if (top > m) {
          alpha = ex2(m - top);                     // 0 while m is -inf
          m = top;
        }
        fresh = __any_sync(kFull, m == -INFINITY);
        weights();
        l *= alpha;
        if (t > 0) {
          // O is rescaled once the product of the tile before is done.  (The
          // barrier is waited on only here: the scores of tile t - 1 followed
          // the product of tile t - 3 and that of tile t + 1 awaits this one's
          // weights, so the phase cannot be mistaken.)
          if (!warp_wait(o_done + 8 * (2 * tile + ((t - 1) & 1)), ((t - 1) >> 1) & 1, s_abort)) {
            done = false;
            break;
          }
          fence_after_sync();
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
    const float v_scale = load_global(a.v_scale);
    // the last product is done: O is complete
    if (done && n_tiles > 0)
      done = warp_wait(o_done + 8 * (2 * tile + ((n_tiles - 1) & 1)), ((n_tiles - 1) >> 1) & 1, s_abort);
    fence_after_sync();
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float lse2 = l == 0.0f ? -INFINITY : m + (log2f(l) - kShift);
    const int64_t part = (token * a.num_heads + q_head) * a.num_splits + split;
    if (done) {                                     // uniform over the warp
      // The rows leave in pieces of 128 bytes (32 fp32 or 64 bf16), eight lanes
      // to a piece, through the shared memory of the warp's query rows, which
      // no product reads any more (each lane storing its own row touches 32
      // lines at a time: 2.2 us a CTA).
      const float f = a.num_splits > 1 ? inv : inv * v_scale;
      const uint32_t stage = bar - S::kMisc + tile * S::kQTile + (lanes >> 9);     // 32 rows of 128 bytes a warp
      const uint64_t mine =
          row >= rows ? 0
          : a.num_splits > 1
              ? reinterpret_cast<uint64_t>(a.part_o + part * D)
              : reinterpret_cast<uint64_t>(static_cast<__nv_bfloat16*>(a.out) + token * a.out_stride_t + q_head * a.out_stride_h);
      uint64_t to[8];                               // of rows 4 i + lane / 8
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int from = 4 * i + (lane >> 3);
        to[i] = static_cast<uint64_t>(__shfl_sync(kFull, static_cast<uint32_t>(mine >> 32), from)) << 32 |
                __shfl_sync(kFull, static_cast<uint32_t>(mine), from);
      }
      auto columns = [&](int c, float (&o)[32]) {
        if (n_tiles > 0) {
          tmem_ld32(o_col + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= f;
      };
      const int pieces = a.num_splits > 1 ? D / 32 : D / 64;
#pragma unroll 1
      for (int c = 0; c < pieces; ++c) {
        float o[32];
        if (a.num_splits > 1) {
          columns(32 * c, o);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared16(stage + sw128_offset(lane, j),
                        make_uint4(__float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]),
                                   __float_as_uint(o[4 * j + 2]), __float_as_uint(o[4 * j + 3])));
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            columns(64 * c + 32 * half, o);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st_shared16(stage + sw128_offset(lane, 4 * half + j),
                          make_uint4(pack_bf16x2(o[8 * j], o[8 * j + 1]), pack_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                     pack_bf16x2(o[8 * j + 4], o[8 * j + 5]), pack_bf16x2(o[8 * j + 6], o[8 * j + 7])));
          }
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
    }
    if (a.num_splits > 1) {
      if (row < rows) a.part_lse[part] = done ? lse2 : __uint_as_float(kAbandoned);
    } else if (row < rows && done && a.lse != nullptr) {
      a.lse[token * a.lse_stride_t + q_head] = lse2 * kLn2;
    }
  } else {
    fewer_registers<S::kOtherRegs>();
    auto have = [&](uint32_t bar, int32_t phase) {
      const bool ok = warp_wait(bar, phase & 1, s_abort);
      fence_after_sync();
      return ok;
    };
    // the warp's products still in flight are drained (bounded, whatever the abort flag says)
    auto drained = [&](uint32_t elected, uint32_t bar) {
      warp_commit(elected, bar);
      const long long start = clock64();
      while (!mbar_try_wait(bar, 0)) {
        if (clock64() - start > kDrainCycles) {
          *s_abort = 1;
          break;
        }
      }
      __syncwarp();
    };
    if (warp < S::kScoreWarp) {
      produce<D, kTiles, false>(a, b, head, keys, s0, n_tiles, warp - S::kSoftmaxWarps, lane,
                                rq.cut && threadIdx.x == 32 * S::kSoftmaxWarps, base, k_full, k_empty,
                                valid_ring, s_abort);
    } else if (warp == S::kScoreWarp) {
      // ---- S_w(t) = Q_w K(t)^T (one elected lane; the warp waits together) -----
      constexpr uint32_t kIdesc = idesc_f16(128, kKeys, false);
      set_up_done();
      const uint32_t tmem = __shfl_sync(kFull, *s_tmem, 0);
      const uint32_t elected = elect_lane();
      const uint64_t qdesc = sw128_desc(base, 16, 1024), kdesc = sw128_desc(base + S::kK, 16, 1024);
      bool ok = n_tiles > 0 && have(q_full, 0);
      for (int32_t t = 0; t < n_tiles && ok; ++t) {
        ok = have(k_full + 8 * (t % S::kStages), t / S::kStages);
        const uint64_t kd = kdesc + (((t % S::kStages) * S::kTileBytes) >> 4);
#pragma unroll
        for (int w = 0; w < kTiles; ++w) {
          // the buffer held the scores, then the weights, of tile t - 2
          if (t >= 2) ok = ok && have(o_done + 8 * (2 * w + (t & 1)), (t >> 1) - 1);
          if (!ok) break;
          const uint64_t qd = qdesc + ((w * S::kQTile) >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            warp_mma(elected, tmem + kSCol + kKeys * (2 * w + (t & 1)),
                     qd + (((ks >> 2) * kBlockBytes + 32 * (ks & 3)) >> 4),
                     kd + (((ks >> 2) * kKBlock + 32 * (ks & 3)) >> 4), kIdesc, ks != 0);
          warp_commit(elected, s_full + 8 * (2 * w + (t & 1)));
          // an arrival of this warp's own too: the masks that the key warps wrote
          // before their tile pass on to the softmax
          if (lane == 0) mbar_arrive(s_full + 8 * (2 * w + (t & 1)));
        }
        if (ok) warp_commit(elected, k_empty + 8 * (t % S::kStages));
      }
      drained(elected, drain);
    } else if (warp < S::kOutputWarp) {
      produce<D, kTiles, true>(a, b, head, keys, s0, n_tiles, warp - S::kScoreWarp - 1, lane, false, base, v_full,
                               v_empty, valid_ring, s_abort);
    } else {
      // ---- O_w += P_w(t) V(t) ---------------------------------------------------
      constexpr uint32_t kIdesc = idesc_f16(128, D, true);
      set_up_done();
      const uint32_t tmem = __shfl_sync(kFull, *s_tmem, 0);
      const uint32_t elected = elect_lane();
      const uint64_t vdesc = sw128_desc(base + S::kV, kKBlock, 1024);
      bool ok = true;
      for (int32_t t = 0; t < n_tiles && ok; ++t) {
#ifdef KVQ_ATTN_STALL_TILE
        // Failure-detection build only (tests/test_gpu_per_head_timeout.py):
        // no product from this tile on, as if the tensor work never
        // completed; the other roles' bounded waits run out.
        if (t == KVQ_ATTN_STALL_TILE) break;
#endif
        ok = have(v_full + 8 * (t % S::kStages), t / S::kStages);
        const uint64_t vd = vdesc + (((t % S::kStages) * S::kTileBytes) >> 4);
#pragma unroll
        for (int w = 0; w < kTiles; ++w) {
          ok = ok && have(p_full + 8 * (2 * w + (t & 1)), t >> 1);
          if (!ok) break;
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks)
            warp_mma_ta(elected, tmem + w * D, tmem + kSCol + kKeys * (2 * w + (t & 1)) + 8 * ks,
                        vd + ((2048 * ks) >> 4), kIdesc, (t > 0 || ks > 0) ? 1u : 0u);
          warp_commit(elected, o_done + 8 * (2 * w + (t & 1)));
        }
        if (ok) warp_commit(elected, v_empty + 8 * (t % S::kStages));
      }
      drained(elected, drain + 8);
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

template <int D, int kTiles>
cudaError_t launch(const PerHeadAttentionArgs& a, cudaStream_t stream) {
  using S = Shape<D, kTiles>;
  const cudaError_t e = cudaFuncSetAttribute(per_head_prefill_kernel<D, kTiles>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (static_cast<int64_t>(a.max_query_len) * a.group + 128 * kTiles - 1) / (128 * kTiles);
  const dim3 grid(static_cast<unsigned>(blocks * a.num_kv_heads * a.num_splits), static_cast<unsigned>(a.batch_size));
  return launch_dependent(per_head_prefill_kernel<D, kTiles>, grid, S::kThreads, S::kSmem, 1, stream, a,
                          static_cast<int32_t>(blocks));
}

}  // namespace

cudaError_t launch_per_head_prefill(const PerHeadAttentionArgs& a, cudaStream_t stream) {
  // two row tiles share a decoded key tile wherever a request can fill them
  const bool two = per_head_prefill_rows(static_cast<int64_t>(a.max_query_len) * a.group, a.head_size) == 256;
  switch (a.head_size) {
    case 64: return two ? launch<64, 2>(a, stream) : launch<64, 1>(a, stream);
    case 128: return two ? launch<128, 2>(a, stream) : launch<128, 1>(a, stream);
    default: return launch<256, 1>(a, stream);       // one tile's O fills the tensor memory
  }
}

}  // namespace kvq
