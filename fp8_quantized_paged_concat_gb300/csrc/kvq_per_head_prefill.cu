// kvq_per_head_prefill.cu -- the attention over the paged per-head NVFP4
// cache (window and tree masks, defined in kvq_per_head_attention.cu) for
// many query rows that share a key head: chunks of new tokens, large draft
// trees.  The products bound it: 4 D flops for each (row, visible key).
//
// Design: one CTA per (block of 128 kTiles query rows, key head, range of
// keys), one CTA per SM; the rows are (token, head) pairs of one request.
// Two row tiles (kTiles = 2) share every decoded key tile, and their softmax
// and products alternate: while one tile's scores become weights, the tensor
// core works on the other tile.
//   - tensor memory: O of tile w in columns [D w, +D); scores S (128 x kKeys
//     fp32) in columns 256 on, one buffer per row tile (two buffers for a
//     single tile); the weights P (f16) overwrite the first half of their S;
//   - shared memory: q in f16 (scaled by each row's power of two), K tiles
//     and V tiles (kKeys x D f16, 128-byte swizzle), two stages each; K is
//     free once its scores are formed, V once its product is;
//   - producer warps decode the entries: 8 lanes take 8 rows of a 64-column
//     block, so that their 16-byte stores fall in different banks; a tile's
//     loads are issued a tile ahead, its page ids two;
//   - one thread issues the products, per key tile t: P_0 V, S_0(t + 1), P_1
//     V, S_1(t + 1) (for a single row tile S(t + 1), then P V(t));
//   - four softmax warps per row tile, one thread per row, in one pass over
//     the scores: the weights are formed against the reference maximum of the
//     tiles before, and only when a score exceeds it by 2^8 is the pass
//     repeated with the new one and O rescaled (after which the row's weights
//     are again at most 1).
// Every wait is bounded; on expiry the CTA records KVQ_STATUS_TIMEOUT, drains
// its products, frees its tensor memory and leaves its rows unwritten.
#include "kvq_per_head_attention.cuh"

namespace kvq {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;
constexpr int kStages = 2;
constexpr int kValidRing = 4;
constexpr uint32_t kBlockBytes = 128 * 128;       // 64 dimensions of 128 rows of q

template <int D, int kTiles>
struct Shape {
  static constexpr int kKeys = D == 256 ? 64 : 128;          // keys per tile
  static constexpr int kSoftmaxWarps = 4 * kTiles;
  static constexpr int kProducers = kTiles == 2 ? 4 : 8;
  static constexpr int kMmaWarp = kSoftmaxWarps + kProducers;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr int kBlocks = D / 64;                     // 64-dimension blocks
  static constexpr uint32_t kKBlock = kKeys * 128;
  static constexpr uint32_t kTileBytes = kBlocks * kKBlock;  // one stage of K or V
  static constexpr uint32_t kQTile = kBlocks * kBlockBytes;
  static constexpr uint32_t kK = kTiles * kQTile;
  static constexpr uint32_t kV = kK + kStages * kTileBytes;
  static constexpr uint32_t kMisc = kV + kStages * kTileBytes;
  // at least 116 KB, so that a second CTA, which would wait for tensor memory, does not share the SM
  static constexpr uint32_t kSmem = kMisc + 512 + 1024 > 116 * 1024 ? kMisc + 512 + 1024 : 116 * 1024;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(kTiles * D <= 256 && 256 + 2 * kKeys <= 512, "tensor memory");
  static constexpr int kPasses = kKeys / (8 * kProducers);   // rows of a tile per producer lane
};

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
  if (d < 0) return static_cast<uint32_t>(__ldg(row) << static_cast<int>(-d));
  const int64_t w = d >> 6;
  const int sh = static_cast<int>(d & 63);
  uint64_t v = w < words ? __ldg(row + w) >> sh : 0;
  if (sh > 32 && w + 1 < words) v |= __ldg(row + w + 1) << (64 - sh);
  return static_cast<uint32_t>(v);
}

// Raw pieces of one tile's rows in a producer lane: 16 (D = 64: 16, 128: 32,
// 256: 64) codes and their scales.
template <int D>
struct Piece {
  static constexpr int kWords = D / 32;              // 32-bit words of codes per lane (8 codes each)
  uint32_t w[kWords];
  uint32_t sf;
};

template <int D>
__device__ __forceinline__ void load_piece(const uint8_t* data, const uint8_t* scales, int k, Piece<D>& e) {
  if constexpr (D == 64) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(data + 8 * k));
    e.w[0] = v.x;
    e.w[1] = v.y;
    e.sf = __ldg(scales + k);
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(data + (D / 8) * k) + i);
      e.w[4 * i] = v.x;
      e.w[4 * i + 1] = v.y;
      e.w[4 * i + 2] = v.z;
      e.w[4 * i + 3] = v.w;
    }
    if constexpr (D == 128)
      e.sf = __ldg(reinterpret_cast<const uint16_t*>(scales + 2 * k));
    else
      e.sf = __ldg(reinterpret_cast<const uint32_t*>(scales + 4 * k));
  }
}

// Decodes a piece and stores its 16-byte chunks into row r of a tile.
template <int D, uint32_t kKBlock, bool kValues>
__device__ __forceinline__ void store_piece(uint32_t tile, uint32_t r, int k, const Piece<D>& e) {
  // a lane's D / 4 dimensions: block (D / 4) k / 64, chunks from ((D / 4) k % 64) / 8 on
  const uint32_t base = tile + (D * k / 256) * kKBlock + r * 128u + ((r & 7u) << 4);
  const uint32_t chunk0 = (D / 32 * k) & 7;
#pragma unroll
  for (int p = 0; p < (D + 127) / 128; ++p) {        // two scales at a time
    uint32_t s2 = bits(e4m3x2_to_half2(e.sf >> (16 * p)));
    if constexpr (kValues) s2 = finite_scales(s2);
#pragma unroll
    for (int j = 0; j < (D == 64 ? 2 : 4); ++j) {
      const uint32_t sf = prmt(s2, s2, j < 2 ? 0x1010 : 0x3232);
      uint32_t h[4];
      e2m1x8(e.w[4 * p + j], h);
      st_shared16(base ^ ((chunk0 + 4 * p + j) << 4),
                  make_uint4(hmul2(h[0], sf), hmul2(h[1], sf), hmul2(h[2], sf), hmul2(h[3], sf)));
    }
  }
}

template <int D, int kTiles>
__global__ void __launch_bounds__(Shape<D, kTiles>::kThreads, 1)
    per_head_prefill_kernel(const PerHeadAttentionArgs a, int32_t row_blocks) {
  using S = Shape<D, kTiles>;
  constexpr int kKeys = S::kKeys;
  // (key head, row block, range): heads vary fastest; the last row blocks of a
  // causal chunk, which see the most keys, come first
  const uint32_t head = blockIdx.x % a.num_kv_heads, rest = blockIdx.x / a.num_kv_heads;
  const int32_t rb = row_blocks - 1 - static_cast<int32_t>(rest % row_blocks), split = rest / row_blocks;
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
  int32_t s0 = 0, s1 = keys.steps;
  if (a.num_splits > 1) {
    const int64_t per = a.split_keys / kKeys;
    s0 = static_cast<int32_t>(min(static_cast<int64_t>(keys.steps), split * per));
    if (split < a.num_splits - 1) s1 = static_cast<int32_t>(min(static_cast<int64_t>(keys.steps), (split + 1) * per));
    if (s0 == s1) {
      // an empty range: it weighs nothing when the ranges are joined
      for (int r = threadIdx.x; r < rows; r += S::kThreads) {
        const uint32_t flat = static_cast<uint32_t>(row0 + r), tk = a.group_div.div(flat);
        const int64_t row = (rq.token0 + tk) * a.num_heads + head * a.group + (flat - tk * a.group);
        a.part_lse[row * a.num_splits + split] = -INFINITY;
      }
      return;
    }
  }
  const int32_t n_tiles = s1 - s0;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t bar = base + S::kMisc;
  const uint32_t k_full = bar, k_empty = bar + 16, v_full = bar + 32, v_empty = bar + 48;   // [kStages] each
  const uint32_t s_full = bar + 64, p_full = bar + 80, o_done = bar + 96;                   // [2] each
  const uint32_t valid_full = bar + 112, drain = bar + 144;                                 // [kValidRing], 1
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + S::kMisc + 160);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + S::kMisc + 164);
  uint8_t* valid_ring = smem + S::kMisc + 256;     // [kValidRing][16]: bit per key of the tile
  static_assert(kStages == 2 && kValidRing == 4, "barrier layout");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(s_tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, S::kProducers);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, S::kProducers);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(o_done + 8 * i, 1);
    }
    for (int i = 0; i < kValidRing; ++i) mbar_init(valid_full + 8 * i, S::kProducers);
    mbar_init(drain, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  const bool is_softmax = warp < S::kSoftmaxWarps;
  const bool is_producer = !is_softmax && warp < S::kMmaWarp;
  const int tile = warp >> 2;                       // softmax: row tile
  const int32_t row = static_cast<int32_t>(threadIdx.x);   // softmax: row of the block

  // ---- softmax threads: their query row -> shared memory ------------------
  float sc = 0.0f;                                  // score -> base-2 exponent
  int64_t token = 0;
  int32_t q_head = 0;
  int32_t pos_hi = -1, pos_lo = 0;
  if (is_softmax) {
    const bool live = row < rows;
    const uint4* src = nullptr;
    float amax = 0.0f;
    if (live) {
      const uint32_t flat = static_cast<uint32_t>(row0 + row), tk = a.group_div.div(flat);
      token = rq.token0 + tk;
      q_head = head * a.group + (flat - tk * a.group);
      const int64_t p = rq.first_pos + tk;
      pos_hi = static_cast<int32_t>(max(int64_t{-1}, min(p, static_cast<int64_t>(rq.len) - 1)));
      pos_lo = a.window > 0 ? static_cast<int32_t>(min(static_cast<int64_t>(rq.len), max(int64_t{0}, p - a.window + 1))) : 0;
      src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + token * a.q_stride_t +
                                           q_head * a.q_stride_h);
#pragma unroll 8
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = __ldg(src + i);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[j])), fabsf(bf16_hi(x[j]))));
      }
    }
    const RowScale rs = row_scale(amax);
    sc = a.scale_log2 * __ldg(a.k_scale) * rs.i[0] * rs.i[1];
    const uint32_t q_tile = base + tile * S::kQTile;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      uint4 v = make_uint4(0, 0, 0, 0);             // rows past the block's are zero
      if (live) {
        const uint4 x = __ldg(src + i);
        v = make_uint4(pack_f16x2(bf16_lo(x.x) * rs.f[0] * rs.f[1], bf16_hi(x.x) * rs.f[0] * rs.f[1]),
                       pack_f16x2(bf16_lo(x.y) * rs.f[0] * rs.f[1], bf16_hi(x.y) * rs.f[0] * rs.f[1]),
                       pack_f16x2(bf16_lo(x.z) * rs.f[0] * rs.f[1], bf16_hi(x.z) * rs.f[0] * rs.f[1]),
                       pack_f16x2(bf16_lo(x.w) * rs.f[0] * rs.f[1], bf16_hi(x.w) * rs.f[0] * rs.f[1]));
      }
      st_shared16(q_tile + (i >> 3) * kBlockBytes + sw128_offset(row & 127, i & 7), v);
    }
    fence_async_smem();
  }

  // ---- producers: the first tile's loads ----------------------------------
  // Lane (k = lane / 8, lane % 8) takes D / 4 dimensions of rows 8 (warp +
  // kProducers i) + lane % 8, i < kPasses.
  const int k = lane >> 3;
  const uint32_t r0 = 8 * (warp - S::kSoftmaxWarps) + (lane & 7);
  bool bad_index = rq.cut && threadIdx.x == 0;
  Piece<D> pk[S::kPasses], pv[S::kPasses];
  int32_t page[S::kPasses], in_page[S::kPasses], next[S::kPasses];   // this tile's pages and rows, the next one's ids
  // page id of key r of tile t: -1 past the range, INT32_MAX for a column past the table or a negative id
  auto page_id = [&](int32_t t, uint32_t r) -> int32_t {
    if (t >= n_tiles) return -1;
    const int32_t p = keys.base(s0 + t) + static_cast<int32_t>(r);
    if (p >= keys.limit(s0 + t)) return -1;
    const uint32_t col = a.block_div.div(static_cast<uint32_t>(p));
    if (col >= static_cast<uint32_t>(a.block_table_width)) return INT32_MAX;
    const int32_t id = __ldg(a.block_table + b * a.block_table_stride + col);
    return id < 0 ? INT32_MAX : id;
  };
  // turns the ids loaded for tile t into pages and rows
  auto resolve = [&](int32_t t) {
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      page[i] = next[i];
      in_page[i] = 0;
      if (page[i] >= a.num_pages) {
        bad_index = true;
        page[i] = -1;
      }
      if (page[i] >= 0) {
        const uint32_t p = keys.base(s0 + t) + r0 + 8 * S::kProducers * i;
        const uint32_t off = p - a.block_div.div(p) * static_cast<uint32_t>(a.block_size);
        in_page[i] = static_cast<int32_t>(off) * a.row_offset + static_cast<int32_t>(head) * a.row_head;
      }
    }
  };
  auto load = [&](int side, Piece<D> (&e)[S::kPasses]) {
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      if (page[i] < 0) {
        e[i] = Piece<D>{};                          // decodes to zeros
        continue;
      }
      const uint8_t* region = a.cache + (static_cast<int64_t>(page[i]) * 2 + side) * a.region;
      load_piece<D>(region + static_cast<int64_t>(in_page[i]) * (D / 2),
                    region + a.scales + static_cast<int64_t>(in_page[i]) * (D / 16), k, e[i]);
    }
  };
  if (is_producer) {
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) next[i] = page_id(0, r0 + 8 * S::kProducers * i);
    resolve(0);
    if (n_tiles > 0) {
      load(0, pk);
      load(1, pv);
    }
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) next[i] = page_id(1, r0 + 8 * S::kProducers * i);
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *s_tmem;

  int mma_issued = 0;
  float m = -INFINITY, l = 0.0f;
  if (is_softmax) {
    // ---- softmax ------------------------------------------------------------
    const uint32_t lanes = (warp & 3) * 32u << 16;
    const uint32_t o_col = tmem + lanes + tile * D;
    for (int32_t t = 0; t < n_tiles; ++t) {
      const int buf = kTiles == 2 ? tile : t & 1;
      const uint32_t s_col = tmem + lanes + kSCol + kKeys * buf;
      // which of the tile's keys the row sees
      const int32_t p0 = keys.base(s0 + t), limit = keys.limit(s0 + t);
      if (!warp_wait_or_abort(valid_full + 8 * (t % kValidRing), (t / kValidRing) & 1, s_abort)) break;
      uint32_t see[kKeys / 32];
      bool all = p0 + kKeys <= limit;
#pragma unroll
      for (int c = 0; c < kKeys / 32; ++c) {
        see[c] = reinterpret_cast<const volatile uint32_t*>(valid_ring + 16 * (t % kValidRing))[c];
        all = all && see[c] == kFull;
      }
      if (a.tree_mask != nullptr)
        all = all && p0 + kKeys <= rq.first_pos;
      else
        all = all && p0 + kKeys - 1 <= pos_hi && (p0 >= pos_lo || p0 + kKeys <= a.num_sinks);
      const bool masked = __any_sync(kFull, !all && row < rows);
      if (masked) {
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c) {
          const int32_t pc = p0 + 32 * c;
          uint32_t w;
          if (row >= rows)
            w = 0;
          else if (a.tree_mask != nullptr)
            w = (rq.first_pos > 0 ? range_bits(pc, 0, static_cast<int32_t>(min(rq.first_pos - 1, int64_t{INT32_MAX} - 64))) : 0u) |
                tree_bits(a.tree_mask + token * a.tree_stride, a.tree_words, pc - rq.first_pos);
          else
            w = range_bits(pc, pos_lo, pos_hi) | range_bits(pc, 0, min(a.num_sinks - 1, pos_hi));
          see[c] &= w;
        }
      }
      if (!warp_wait_or_abort(s_full + 8 * buf, (kTiles == 2 ? t : t >> 1) & 1, s_abort)) break;
      fence_after_sync();

      uint32_t p[kKeys / 2];
      float top, sum;
      // weights against the reference m: p, their sum, and the largest exponent
      auto pass = [&](float off) {
        float2 sums[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c) {
          float s[32];
          tmem_ld32(s_col + 32 * c, s);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 z = ffma2(make_float2(s[i], s[i + 1]), make_float2(sc, sc), make_float2(off, off));
            if (masked) {
              z.x = (see[c] >> i) & 1 ? z.x : -INFINITY;
              z.y = (see[c] >> (i + 1)) & 1 ? z.y : -INFINITY;
            }
            tops[(i >> 1) & 3] = fmax3(tops[(i >> 1) & 3], z.x, z.y);
            const float2 w = make_float2(ex2(z.x), ex2(z.y));
            sums[(i >> 1) & 1] = fadd2(sums[(i >> 1) & 1], w);
            p[16 * c + (i >> 1)] = pack_f16x2(w.x, w.y);
          }
        }
        const float2 both = fadd2(sums[0], sums[1]);
        sum = both.x + both.y;
        top = fmaxf(fmax3(tops[0], tops[1], tops[2]), tops[3]);
      };
      const float m_use = m == -INFINITY ? 0.0f : m;
      pass(kShift - m_use);
      const bool grow = top > -INFINITY && (m == -INFINITY || top > kShift + kGrow);
      float alpha = 1.0f;
      if (__any_sync(kFull, grow)) {
        if (grow) {
          const float m_new = top - kShift + m_use;
          alpha = ex2(m - m_new);                   // 0 while m is -inf
          m = m_new;
        }
        pass(kShift - (m == -INFINITY ? 0.0f : m));
      }
      l = l * alpha + sum;
      // the product of the tile before is done: O may be rescaled (and the
      // barrier's phases stay in step)
      if (t > 0 && !warp_wait_or_abort(o_done + 8 * (kTiles == 2 ? tile : 0), (t - 1) & 1, s_abort)) break;
      if (t > 0 && __any_sync(kFull, alpha != 1.0f)) {
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
#pragma unroll
      for (int c = 0; c < kKeys / 32; ++c) tmem_st16(s_col + 16 * c, p + 16 * c);
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + 8 * (kTiles == 2 ? tile : 0));
    }
  } else if (is_producer) {
    // ---- producers ----------------------------------------------------------
    for (int32_t t = 0; t < n_tiles; ++t) {
      const int st = t % kStages;
      // which keys exist, for the softmax (the ring slot's last reader was
      // four tiles ago: scores of tile t - 2, whose buffer K(t) takes, exist
      // only once the weights of tile t - 4 were used)
#pragma unroll
      for (int i = 0; i < S::kPasses; ++i) {
        const uint32_t have = __ballot_sync(kFull, page[i] >= 0);
        if (lane == 0) valid_ring[16 * (t % kValidRing) + (r0 >> 3) + S::kProducers * i] = static_cast<uint8_t>(have);
      }
      if (t >= kStages && !warp_wait_or_abort(k_empty + 8 * st, (t / kStages - 1) & 1, s_abort)) break;
#pragma unroll
      for (int i = 0; i < S::kPasses; ++i)
        store_piece<D, S::kKBlock, false>(base + S::kK + st * S::kTileBytes, r0 + 8 * S::kProducers * i, k, pk[i]);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(valid_full + 8 * (t % kValidRing));
        mbar_arrive(k_full + 8 * st);
      }
      if (t + 1 < n_tiles) {
        resolve(t + 1);
        load(0, pk);
#pragma unroll
        for (int i = 0; i < S::kPasses; ++i) next[i] = page_id(t + 2, r0 + 8 * S::kProducers * i);
      }
      if (t >= kStages && !warp_wait_or_abort(v_empty + 8 * st, (t / kStages - 1) & 1, s_abort)) break;
#pragma unroll
      for (int i = 0; i < S::kPasses; ++i)
        store_piece<D, S::kKBlock, true>(base + S::kV + st * S::kTileBytes, r0 + 8 * S::kProducers * i, k, pv[i]);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full + 8 * st);
      if (t + 1 < n_tiles) load(1, pv);
    }
  } else if (lane == 0) {
    // ---- products (one thread) ----------------------------------------------
    constexpr uint32_t kIdescS = idesc_f16(128, kKeys, false);
    constexpr uint32_t kIdescO = idesc_f16(128, D, true);
    const uint64_t qdesc = sw128_desc(base, 16, 1024);
    const uint64_t kdesc = sw128_desc(base + S::kK, 16, 1024);
    const uint64_t vdesc = sw128_desc(base + S::kV, S::kKBlock, 1024);
    auto scores = [&](int32_t t, int w) {           // S of row tile w (K is there)
      const int st = t % kStages, buf = kTiles == 2 ? w : t & 1;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        mma_bf16(tmem + kSCol + kKeys * buf,
                 qdesc + ((w * S::kQTile + (ks >> 2) * kBlockBytes + 32 * (ks & 3)) >> 4),
                 kdesc + ((st * S::kTileBytes + (ks >> 2) * S::kKBlock + 32 * (ks & 3)) >> 4), kIdescS, ks != 0);
      mma_commit(s_full + 8 * buf);
      mma_issued = 1;
    };
    auto outputs = [&](int32_t t, int w) {          // O of row tile w += P V(t)
      const int st = t % kStages, buf = kTiles == 2 ? w : t & 1;
#pragma unroll
      for (int ks = 0; ks < kKeys / 16; ++ks)
        mma_bf16_ta(tmem + w * D, tmem + kSCol + kKeys * buf + 8 * ks, vdesc + ((st * S::kTileBytes + 2048 * ks) >> 4),
                    kIdescO, (t > 0 || ks > 0) ? 1u : 0u);
    };
    auto have_k = [&](int32_t t) { return wait_or_abort(k_full + 8 * (t % kStages), (t / kStages) & 1, s_abort); };
    auto have_v = [&](int32_t t) { return wait_or_abort(v_full + 8 * (t % kStages), (t / kStages) & 1, s_abort); };
    if (n_tiles > 0 && have_k(0)) {
      fence_after_sync();
#pragma unroll
      for (int w = 0; w < kTiles; ++w) scores(0, w);
      mma_commit(k_empty);
      for (int32_t t = 0; t < n_tiles; ++t) {
        if constexpr (kTiles == 1) {
          if (t + 1 < n_tiles) {
            if (!have_k(t + 1)) break;
            fence_after_sync();
            scores(t + 1, 0);
            mma_commit(k_empty + 8 * ((t + 1) % kStages));
          }
          if (!have_v(t) || !wait_or_abort(p_full, t & 1, s_abort)) break;
          fence_after_sync();
          outputs(t, 0);
          mma_commit(v_empty + 8 * (t % kStages));
          mma_commit(o_done);
        } else {
          bool ok = have_v(t);
#pragma unroll
          for (int w = 0; w < 2 && ok; ++w) {
            ok = wait_or_abort(p_full + 8 * w, t & 1, s_abort);
            if (!ok) break;
            fence_after_sync();
            outputs(t, w);
            if (w == 1) mma_commit(v_empty + 8 * (t % kStages));
            mma_commit(o_done + 8 * w);
            if (t + 1 < n_tiles) {
              if (w == 0) {
                ok = have_k(t + 1);
                if (!ok) break;
                fence_after_sync();
              }
              scores(t + 1, w);
              if (w == 1) mma_commit(k_empty + 8 * ((t + 1) % kStages));
            }
          }
          if (!ok) break;
        }
      }
    }
  }

  // Every role has left its loop: drain the products still in flight.
  fence_before_sync();
  const bool any_mma = __syncthreads_or(mma_issued) != 0;
  fence_after_sync();
  bool aborted = *s_abort != 0;
  if (any_mma) {
    if (threadIdx.x == S::kMmaWarp * 32) mma_commit(drain);
    const long long start = clock64();
    while (!mbar_try_wait(drain, 0)) {              // bounded, ignores the abort flag
      if (clock64() - start > kDrainCycles) {
        aborted = true;
        break;
      }
    }
  }
  fence_after_sync();
  if (bad_index) report(a.status, KVQ_STATUS_BAD_INDEX);
  aborted = __syncthreads_or(aborted) != 0;
  if (aborted && threadIdx.x == 0) report(a.status, KVQ_STATUS_TIMEOUT);

  if (is_softmax) {
    const bool live = row < rows && !aborted;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float lse2 = l == 0.0f ? -INFINITY : m + (log2f(l) - kShift);
    const int64_t part = (token * a.num_heads + q_head) * a.num_splits + split;
    const float f = a.num_splits > 1 ? inv : inv * __ldg(a.v_scale);
    const uint32_t o_col = tmem + ((warp & 3) * 32u << 16) + tile * D;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      float o[32];
      if (n_tiles > 0 && !aborted) {                // uniform over the CTA
        tmem_ld32(o_col + 32 * c, o);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0.0f;
      }
      if (live && a.num_splits > 1) {
        float4* dst = reinterpret_cast<float4*>(a.part_o + part * D + 32 * c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[i] = make_float4(o[4 * i] * f, o[4 * i + 1] * f, o[4 * i + 2] * f, o[4 * i + 3] * f);
      } else if (live) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + token * a.out_stride_t +
                                              q_head * a.out_stride_h + 32 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[i] = make_uint4(pack_bf16x2(o[8 * i] * f, o[8 * i + 1] * f), pack_bf16x2(o[8 * i + 2] * f, o[8 * i + 3] * f),
                              pack_bf16x2(o[8 * i + 4] * f, o[8 * i + 5] * f),
                              pack_bf16x2(o[8 * i + 6] * f, o[8 * i + 7] * f));
      }
      __syncwarp();                                 // the next load is the whole warp's
    }
    if (a.num_splits > 1) {
      if (row < rows) a.part_lse[part] = aborted ? __uint_as_float(kAbandoned) : lse2;
    } else if (live && a.lse != nullptr) {
      a.lse[token * a.lse_stride_t + q_head] = lse2 * kLn2;
    }
  }

  fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kTmemCols) : "memory");
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
  per_head_prefill_kernel<D, kTiles><<<grid, S::kThreads, S::kSmem, stream>>>(a, static_cast<int32_t>(blocks));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_per_head_prefill(const PerHeadAttentionArgs& a, cudaStream_t stream) {
  // two row tiles share a decoded key tile wherever a request can fill them
  const bool two = static_cast<int64_t>(a.max_query_len) * a.group > 128;
  switch (a.head_size) {
    case 64: return two ? launch<64, 2>(a, stream) : launch<64, 1>(a, stream);
    case 128: return two ? launch<128, 2>(a, stream) : launch<128, 1>(a, stream);
    default: return launch<256, 1>(a, stream);       // one tile's O fills the tensor memory
  }
}

}  // namespace kvq
