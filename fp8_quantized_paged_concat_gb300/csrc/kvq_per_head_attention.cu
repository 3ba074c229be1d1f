// kvq_per_head_attention.cu -- attention read straight from the paged
// per-head NVFP4 K/V cache, for grouped query heads, in two forms of mask:
//   window  causal, with a sliding window and a few first tokens that stay
//           visible: the query at position p sees key j iff j <= p and
//           (window <= 0 or j > p - window or j < num_sinks);
//   tree    drafted tokens at the end of the sequence: draft i sees the whole
//           context before the drafts, and draft j iff bit j of its mask.
// For query row (token t, head h) over its visible keys j of key head h /
// group, with k_j, v_j the decoded entries (e2m1 * e4m3, exact):
//   s_j = softmax_scale * k_scale * (q . k_j)
//   out = v_scale * sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  lse = m + ln sum
// (no visible key: out = 0, lse = -inf).
//
// Few query rows (decode): the keys' bytes bound it, 9/16 byte per value.
// One CTA of four warps per (block of 8 kRowTiles query rows, key head, range
// of keys); the rows are (token, head) pairs of one request that share the
// key head.  Each warp takes every fourth step of 32 keys, with its own
// running maximum and sum, and the warps join at the end through shared
// memory; the ranges of a small call run as a cluster and join through its
// distributed shared memory (one request, window of 1024, 64 heads: 7.1 us,
// 7.6 through a workspace and a second launch, 10.4 unsplit), others in a
// second launch.  A warp
// copies a step's raw bytes
// (32 entries of 9 D / 16 bytes, K and V) into its own two-stage ring with
// asynchronous copies, a step ahead, so that nothing but the warp's own
// copies is ever waited for.
//
// The products run as S^T = K Q^T and O^T = V^T P^T on the warp's matrix
// instruction (16 x 8 x 16, f16 in, fp32 sums): the keys (the head
// dimensions) fill the 16-wide side, the query rows only an 8-wide one, so a
// single token's 4 or 8 grouped heads waste little.  Every operand register
// is decoded where it is used: for K, a lane's 16-byte piece of an entry is
// D / 4 whole dimensions of one key; for V, a lane takes D / 8 dimensions of
// four keys and merges two keys' nibbles into one byte before converting it,
// so that a converted pair holds two keys.  The order of the dimensions and
// of the keys inside the products is free, and chosen so that these pieces
// are contiguous; q is loaded in the same order.  P^T comes from S^T by the
// 8 x 8 transposing move.
// f16 holds the decoded entries exactly (at most 6 significant bits, 2^-10 to
// 2688).  A query row is scaled by the power of two that brings its largest
// value to [2^14, 2^15): bf16's 8 bits stay exact in f16 down to 2^-28 of
// that largest value, and what is lost below is under 2^-39 of it.  The
// weights are kept as 2^(s - m + 6) with m at most 2^8 behind the true
// maximum (so <= 2^14) and rounded to f16 (relative 2^-11), the type that the
// matrix instruction takes beside the entries' own: fp32 operands would go
// through tf32 at half the rate with no more mantissa, bf16 would lose eight
// times as much, and the result's bf16 rounding (2^-8) hides it (the measured
// cases' error against 64 bits is 0.00167 of the largest value with it, 0.00166
// in fp32).  Their sum is taken before the rounding, in fp32.
//
// Measured: 128 requests x 4100 keys x 32 heads (8 key heads) of 128, 606 MB:
// 115 us, 5.3 TB/s; about 640 warp instructions per step of 32 keys for 4
// rows, and their issue, not the copies, sets the pace (3 stages or 5 CTAs an
// SM are slower: registers).
#include "kvq_per_head_attention.cuh"
#include "kvq_per_head_plan.h"

namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;                   // keys per warp step
constexpr int kStages = 2;

// Shared memory of one warp's stage: 32 data rows of K, of V, then their scale rows.
template <int D>
struct Stage {
  static constexpr int kRow = D / 2, kScales = D / 16;
  static constexpr int kV = kStep * kRow, kKs = 2 * kStep * kRow, kVs = kKs + kStep * kScales;
  static constexpr int kBytes = kVs + kStep * kScales;
};

// D += A B, A 16 x 16 (row), B 16 x 8 (col), f16 in, fp32 out.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of a b16 fragment held across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Stage row of the key with index n (0..7) inside an 8-key half: the rows of
// keys 2c differ mod 4 over c, and those of 2c and 2c + 1 in parity, which
// keeps the lanes' shared-memory reads apart.
__device__ __forceinline__ uint32_t key_row(uint32_t n) { return (n & 1) ? 4 + ((n >> 1) ^ 1) : n >> 1; }
// 16-byte chunk swizzles of the staged data rows.
template <int D>
__device__ __forceinline__ uint32_t k_chunk(uint32_t row, uint32_t chunk) {
  return D == 256 ? chunk ^ (row & 1) : chunk;
}
template <int D>
__device__ __forceinline__ uint32_t v_chunk(uint32_t row, uint32_t chunk) {
  return D == 256 ? chunk ^ ((row & 3) << 1) : D == 128 ? chunk ^ (row & 2) : chunk;
}

// Distributed shared memory of a cluster: the address in CTA `rank`'s shared
// memory that corresponds to `addr` in one's own, loads from there, and the
// cluster's barrier (also for the shared memory before and after it).
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The ranges of a cluster joined: CTA `rank` of num_splits takes its share of
// the (row, 8 dimensions) of the block.  In every CTA `o` holds the rows' fp32
// sums (rows `stride` bytes apart), `m` and `l` their reference maxima and
// denominators.  Every thread of the cluster comes here.
__device__ __forceinline__ void join_cluster(const PerHeadAttentionArgs& a, const Request& rq, uint32_t kv_head,
                                             int64_t row0, int32_t rows, int32_t rank, int32_t dims, uint32_t o,
                                             uint32_t stride, uint32_t m, uint32_t l) {
  const float v_scale = load_global(a.v_scale);
  cluster_sync();
  const int32_t chunks = dims / 8;
  // (distributed shared memory gives an SM about 14 bytes a clock: the shares are equal)
  for (int32_t i = rank + threadIdx.x * a.num_splits; i < rows * chunks; i += a.num_splits * blockDim.x) {
    const int32_t r = i / chunks, d = (i - r * chunks) * 8;
    // every load is issued before the first is used
    constexpr int kMax = KVQ_PER_HEAD_CLUSTER_SPLITS;
    float ms[kMax], ls[kMax];
    float4 u[kMax], w[kMax];
#pragma unroll
    for (int32_t s = 0; s < kMax; ++s) {
      ms[s] = -INFINITY;
      ls[s] = 0.0f;
      u[s] = w[s] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (s < a.num_splits) {
        ms[s] = cluster_load(cluster_addr(m + 4 * r, s));
        ls[s] = cluster_load(cluster_addr(l + 4 * r, s));
        const uint32_t at = cluster_addr(o + r * stride + 4 * d, s);
        u[s] = cluster_load4(at);
        w[s] = cluster_load4(at + 16);
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int32_t s = 0; s < kMax; ++s) top = fmaxf(top, ms[s]);
    float sum = 0.0f, acc[8] = {};
#pragma unroll
    for (int32_t s = 0; s < kMax; ++s) {
      const float f = ms[s] == -INFINITY ? 1.0f : ex2(ms[s] - top);  // a range that saw nothing holds zeros
      sum += f * ls[s];
      acc[0] += f * u[s].x; acc[1] += f * u[s].y; acc[2] += f * u[s].z; acc[3] += f * u[s].w;
      acc[4] += f * w[s].x; acc[5] += f * w[s].y; acc[6] += f * w[s].z; acc[7] += f * w[s].w;
    }
    const RowAt at = row_at(a, rq, kv_head, static_cast<uint32_t>(row0 + r));
    const float f = (sum == 0.0f ? 0.0f : 1.0f / sum) * v_scale;
    st16(static_cast<__nv_bfloat16*>(a.out) + at.token * a.out_stride_t + at.head * a.out_stride_h + d,
         make_uint4(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f),
                    pack_bf16x2(acc[4] * f, acc[5] * f), pack_bf16x2(acc[6] * f, acc[7] * f)));
    if (d == 0 && a.lse != nullptr)
      a.lse[at.token * a.lse_stride_t + at.head] = sum == 0.0f ? -INFINITY : (top + (log2f(sum) - kShift)) * kLn2;
  }
  cluster_sync();                                // no CTA leaves while its memory is read
}

template <int D, int kRowTiles>
__global__ void __launch_bounds__(kThreads, D == 256 ? 2 : kRowTiles == 2 ? 3 : 4)
    per_head_attention_kernel(const PerHeadAttentionArgs a, int32_t row_blocks) {
  using St = Stage<D>;
  constexpr int kRows = 8 * kRowTiles;
  constexpr int kKSteps = D / 16;                // 16-dimension steps of K Q^T
  constexpr int kDimTiles = D / 16;              // 16-dimension tiles of V^T P^T
  wait_for_previous();
  const Place place = place_of(a, row_blocks);
  const uint32_t head = place.head;
  const int32_t rb = place.row_block, split = place.split;
  const int b = blockIdx.y;
  Request rq;
  if (!request_of(a, b, rq)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, KVQ_STATUS_BAD_BATCH);
    return;
  }
  const int64_t total_rows = static_cast<int64_t>(rq.tokens) * a.group;
  const int64_t row0 = static_cast<int64_t>(rb) * kRows;
  if (row0 >= total_rows) return;
  const int32_t rows = static_cast<int32_t>(min(static_cast<int64_t>(kRows), total_rows - row0));
  const int32_t t0 = a.group_div.div(static_cast<uint32_t>(row0));
  const int32_t t1 = a.group_div.div(static_cast<uint32_t>(row0 + rows - 1));
  const Keys<kStep> keys = keys_of<kStep>(a, rq, t0, t1);
  int32_t s0, s1;
  range_of(a, keys, split, s0, s1);

  allow_dependents();
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * St::kBytes);

  // ---- asynchronous copies -------------------------------------------------
  // Lane l looks up key l of a step: page id, loaded a step before the copies
  // that use it start and looked at only there, address, scale copies; the
  // data rows are copied 16 bytes a lane, kLanes lanes to a row.
  const int32_t* table = a.block_table + b * a.block_table_stride;
  const uint32_t head_row = head * static_cast<uint32_t>(a.row_head);
  bool bad_index = rq.cut && threadIdx.x == 0;
  LookUp next;                                   // the lane's key of the next step to be copied
  auto look_up = [&](int32_t step) {
    const uint32_t p = static_cast<uint32_t>(keys.base(step)) + lane;
    next = look_up_position(a, table, head_row, step < s1 && p < static_cast<uint32_t>(keys.limit(step)), p);
  };
  // one group of copies (empty past the range); returns the step's keys that exist
  auto start = [&](int32_t step, int stage) -> uint32_t {
    uint32_t there = 0;
    if (step < s1) {
      const bool ok = next.in && next.id >= 0 && next.id < a.num_pages;
      bad_index = bad_index || (next.in && !ok);
      there = __ballot_sync(kFull, ok);
      const uint8_t* page = at_offset(a.cache, ok ? next.id : 0, 2 * a.region);   // some page where there is none
      const uint32_t row = ok ? next.row : 0;
      const uint32_t st = ring + stage * St::kBytes;
      const uint8_t* scales = at_offset(page + a.scales, row, St::kScales);
      cp_async<St::kScales>(st + St::kKs + lane * St::kScales, scales, ok ? St::kScales : 0);
      cp_async<St::kScales>(st + St::kVs + lane * St::kScales, scales + a.region, ok ? St::kScales : 0);
      const uint64_t data = reinterpret_cast<uint64_t>(at_offset(page, row, St::kRow));
      constexpr int kLanes = St::kRow / 16;      // lanes that copy one data row
#pragma unroll
      for (int it = 0; it < kLanes; ++it) {
        const int key = it * (32 / kLanes) + lane / kLanes;
        const uint32_t chunk = lane % kLanes;
        const uint64_t at = static_cast<uint64_t>(__shfl_sync(kFull, static_cast<uint32_t>(data >> 32), key)) << 32 |
                            __shfl_sync(kFull, static_cast<uint32_t>(data), key);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(at) + 16 * chunk;
        const uint32_t k_dst = st + key * St::kRow + 16 * k_chunk<D>(key, chunk);
        const uint32_t v_dst = st + St::kV + key * St::kRow + 16 * v_chunk<D>(key, chunk);
        const uint32_t n = (there >> key) & 1 ? 16 : 0;
        cp_async<16>(k_dst, src, n);
        cp_async<16>(v_dst, src + a.region, n);
      }
    }
    cp_commit();
    return there;
  };
  // this warp's steps: first, first + kWarps, ...
  const int32_t first = s0 + warp;
  uint32_t valid_ring[kStages - 1];              // of the steps in flight: bit i = key i exists
  look_up(first);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    valid_ring[i] = start(first + i * kWarps, i);
    look_up(first + (i + 1) * kWarps);
  }

  // ---- the query rows ------------------------------------------------------
  // Lane (g, c) holds dimensions [c D/4, +D/4) of row 8 nt + g, scaled by a
  // power of two; the score of row 2c + x is multiplied back by sc.
  uint32_t q[kRowTiles][kKSteps][2];
  float sc[kRowTiles][2];
  float m[kRowTiles][2], l[kRowTiles][2];                 // reference maximum, sum
  const float scale = a.scale_log2 * load_global(a.k_scale);
#pragma unroll
  for (int nt = 0; nt < kRowTiles; ++nt) {
    const int32_t r = 8 * nt + g;
    float amax = 0.0f;
    uint4 w[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) w[i] = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      const uint32_t flat = static_cast<uint32_t>(row0 + r), tk = a.group_div.div(flat);
      const int32_t h = head * a.group + (flat - tk * a.group);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                        (rq.token0 + tk) * a.q_stride_t + h * a.q_stride_h + c * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        w[i] = load_global(src + i);
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[j])), fabsf(bf16_hi(x[j]))));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    const RowScale rs = row_scale(amax);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[nt][2 * i + (j >> 1)][j & 1] = pack_f16x2(bf16_lo(x[j]) * rs.f[0] * rs.f[1], bf16_hi(x[j]) * rs.f[0] * rs.f[1]);
    }
    const float back = scale * rs.i[0] * rs.i[1];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      // row 2c + x of the tile is loaded by the lanes with g = 2c + x
      sc[nt][x] = __shfl_sync(kFull, back, (2 * c + x) * 4);
      if (sc[nt][x] == 0.0f) sc[nt][x] = 1e-30f;            // as good as 0 for any score, but 0 for no infinity
      const int32_t rr = 8 * nt + 2 * c + x;
      m[nt][x] = rr < rows ? -INFINITY : 0.0f;
      l[nt][x] = 0.0f;
    }
  }
  // a step inside these positions is visible to every row
  const int32_t all_hi = static_cast<int32_t>(max(int64_t{-1}, rq.first_pos + (a.tree_mask ? -1 : t0)));
  const int32_t all_lo =
      a.tree_mask == nullptr && a.window > 0 ? static_cast<int32_t>(max(int64_t{0}, rq.first_pos + t1 - a.window + 1)) : 0;

  float o[kDimTiles][kRowTiles][4];
#pragma unroll
  for (int t = 0; t < kDimTiles; ++t)
#pragma unroll
    for (int nt = 0; nt < kRowTiles; ++nt) o[t][nt][0] = o[t][nt][1] = o[t][nt][2] = o[t][nt][3] = 0.0f;

  const uint32_t rg = key_row(g), r0 = key_row(2 * c), r1 = key_row(2 * c + 1);
  int stage = 0;
  for (int32_t step = first; step < s1; step += kWarps) {
    cp_wait<kStages - 2>();
    __syncwarp();                                // the step has landed, and the stage before it has been read
    const uint32_t valid = valid_ring[0];
#pragma unroll
    for (int i = 0; i + 2 < kStages; ++i) valid_ring[i] = valid_ring[i + 1];
    valid_ring[kStages - 2] = start(step + (kStages - 1) * kWarps, stage == 0 ? kStages - 1 : stage - 1);
    look_up(step + kStages * kWarps);
    const uint32_t st = ring + stage * St::kBytes;
    stage = stage + 1 == kStages ? 0 : stage + 1;

    // ---- S^T = K Q^T -------------------------------------------------------
    float s[2][kRowTiles][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int nt = 0; nt < kRowTiles; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.0f;
      const uint32_t ra = 16 * mt + rg, rb2 = ra + 8;
      const uint32_t ka = st + ra * St::kRow, kb = st + rb2 * St::kRow;
      // the lane's D / 64 scales of each row
      uint32_t sa, sb;
      if constexpr (D == 64) {
        sa = lds8(st + St::kKs + ra * 4 + c) * 0x0101u;
        sb = lds8(st + St::kKs + rb2 * 4 + c) * 0x0101u;
      } else if constexpr (D == 128) {
        sa = lds16(st + St::kKs + ra * 8 + 2 * c);
        sb = lds16(st + St::kKs + rb2 * 8 + 2 * c);
      } else {
        sa = lds32(st + St::kKs + ra * 16 + 4 * c);
        sb = lds32(st + St::kKs + rb2 * 16 + 4 * c);
      }
#pragma unroll
      for (int i = 0; i < (D + 127) / 128; ++i) {       // 32 dimensions (16 at D = 64) at a time
        uint32_t wa[4], wb[4];
        if constexpr (D == 64) {
          const uint2 x = lds64(ka + 8 * c), y = lds64(kb + 8 * c);
          wa[0] = x.x; wa[1] = x.y; wb[0] = y.x; wb[1] = y.y;
        } else {
          const uint32_t chunk = D == 256 ? 2 * c + i : c;
          const uint4 x = ld_shared16(ka + 16 * k_chunk<D>(ra, chunk)), y = ld_shared16(kb + 16 * k_chunk<D>(rb2, chunk));
          wa[0] = x.x; wa[1] = x.y; wa[2] = x.z; wa[3] = x.w;
          wb[0] = y.x; wb[1] = y.y; wb[2] = y.z; wb[3] = y.w;
        }
        const uint32_t fa = bits(e4m3x2_to_half2(sa >> (16 * i))), fb = bits(e4m3x2_to_half2(sb >> (16 * i)));
#pragma unroll
        for (int j = 0; j < (D == 64 ? 2 : 4); ++j) {   // 8 dimensions: two 16-wide product steps
          // (the broadcast of one half is an operand modifier of the product)
          const uint32_t sfa = (j >> 1) && D != 64 ? high_both(fa) : low_both(fa);
          const uint32_t sfb = (j >> 1) && D != 64 ? high_both(fb) : low_both(fb);
          uint32_t ha[4], hb[4];
          e2m1x8(wa[j], ha);
          e2m1x8(wb[j], hb);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t a0 = hmul2(ha[2 * e], sfa), a1 = hmul2(hb[2 * e], sfb);
            const uint32_t a2 = hmul2(ha[2 * e + 1], sfa), a3 = hmul2(hb[2 * e + 1], sfb);
            const int ks = (D == 64 ? 2 : 4) * 2 * i + 2 * j + e;
#pragma unroll
            for (int nt = 0; nt < kRowTiles; ++nt) mma_f16(s[mt][nt], a0, a1, a2, a3, q[nt][ks][0], q[nt][ks][1]);
          }
        }
      }
    }

    // ---- weights -----------------------------------------------------------
    // s[mt][nt][2 y + x]: key 16 mt + 8 y + key_row(g), query row 8 nt + 2 c + x
    const int32_t base = keys.base(step);
    const bool all = valid == kFull && base + kStep - 1 <= all_hi && (base >= all_lo || base + kStep <= a.num_sinks);
    if (!all) {
#pragma unroll
      for (int nt = 0; nt < kRowTiles; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int32_t rr = 8 * nt + 2 * c + x;
          const int32_t tk = static_cast<int32_t>(a.group_div.div(static_cast<uint32_t>(row0 + min(rr, rows - 1))));
          const int64_t at = rq.first_pos + tk;            // the row's position
          const int32_t hi = rr < rows ? static_cast<int32_t>(max(int64_t{-1}, at)) : -1;
          const int32_t lo = a.window > 0 ? static_cast<int32_t>(max(int64_t{0}, at - a.window + 1)) : 0;
          const float hidden = sc[nt][x] < 0.0f ? INFINITY : -INFINITY;   // the score whose scaled value is -inf
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t i = 8 * e + rg, p = base + i;    // e = 2 mt + y
            bool see = (valid >> i) & 1;
            if (a.tree_mask == nullptr) {
              see = see && p <= hi && (p >= lo || p < a.num_sinks);
            } else if (see && p >= rq.first_pos) {
              const int32_t d = static_cast<int32_t>(p - rq.first_pos);
              const uint64_t* word = a.tree_mask + (rq.token0 + tk) * a.tree_stride + (d >> 6);
              see = (d >> 6) < a.tree_words &&
                    (((kRowTiles == 2 ? load_global64(word) : load_global(word)) >> (d & 63)) & 1);
            }
            if (!see) s[e >> 1][nt][2 * (e & 1) + x] = hidden;
          }
        }
    }
    // Weights against the reference m, the maximum of steps before: no
    // maximum of their own is taken unless their sum shows that one of them
    // may exceed it by 2^kGrow (or there is no reference yet).
    float2 w[kRowTiles][4], sum[kRowTiles];
    auto weights = [&]() {
#pragma unroll
      for (int nt = 0; nt < kRowTiles; ++nt) {
        const float2 off = make_float2(kShift - (m[nt][0] == -INFINITY ? 0.0f : m[nt][0]),
                                       kShift - (m[nt][1] == -INFINITY ? 0.0f : m[nt][1]));
        sum[nt] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float* v = &s[e >> 1][nt][2 * (e & 1)];
          const float2 z = ffma2(make_float2(v[0], v[1]), make_float2(sc[nt][0], sc[nt][1]), off);
          w[nt][e] = make_float2(ex2(z.x), ex2(z.y));
          sum[nt] = fadd2(sum[nt], w[nt][e]);
        }
      }
    };
    weights();
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < kRowTiles; ++nt)
      grow = grow || sum[nt].x > kMaxWeight || sum[nt].y > kMaxWeight || m[nt][0] == -INFINITY || m[nt][1] == -INFINITY;
    if (__any_sync(kFull, grow)) {
#pragma unroll
      for (int nt = 0; nt < kRowTiles; ++nt) {
        float alpha[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, s[e >> 1][nt][2 * (e & 1) + x] * sc[nt][x]);
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
          alpha[x] = 1.0f;
          if (top > m[nt][x]) {
            alpha[x] = ex2(m[nt][x] - top);      // 0 while m is -inf
            m[nt][x] = top;
          }
          l[nt][x] *= alpha[x];
        }
#pragma unroll
        for (int t = 0; t < kDimTiles; ++t) {
          o[t][nt][0] *= alpha[0];
          o[t][nt][1] *= alpha[1];
          o[t][nt][2] *= alpha[0];
          o[t][nt][3] *= alpha[1];
        }
      }
      weights();
    }
    uint32_t p[2][kRowTiles][2];                 // P^T, keys 2c, 2c + 1 and 8 on, of query row g
#pragma unroll
    for (int nt = 0; nt < kRowTiles; ++nt) {
      l[nt][0] += sum[nt].x;
      l[nt][1] += sum[nt].y;
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e >> 1][nt][e & 1] = transpose8(pack_f16x2(w[nt][e].x, w[nt][e].y));
    }

    // ---- O^T += V^T P^T ----------------------------------------------------
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      // keys 2c and 2c + 1 (rows x0, x1) and the two 8 keys on (y0, y1)
      const uint32_t x0 = 16 * mt + r0, x1 = 16 * mt + r1, y0 = x0 + 8, y1 = x1 + 8;
      const uint32_t vs = st + St::kVs, vd = st + St::kV;
#pragma unroll
      for (int i = 0; i < (D == 256 ? 2 : 1); ++i) {    // one scale group (16 dimensions; 8 at D = 64) at a time
        const uint32_t so = D == 64 ? g >> 1 : D == 128 ? g : 2 * g + i;
        uint32_t sx = bits(e4m3x2_to_half2(lds8(vs + x0 * St::kScales + so) | lds8(vs + x1 * St::kScales + so) << 8));
        uint32_t sy = bits(e4m3x2_to_half2(lds8(vs + y0 * St::kScales + so) | lds8(vs + y1 * St::kScales + so) << 8));
        if (!all) {                              // else no entry of the step is hidden from any row
          sx = finite_scales(sx);
          sy = finite_scales(sy);
        }
        uint32_t w[4][2];
        auto load = [&](uint32_t row, uint32_t (&d)[2]) {
          if constexpr (D == 64) {
            d[0] = lds32(vd + row * St::kRow + 4 * g);
          } else {
            const uint32_t at = D == 128 ? 8 * g : 16 * g + 8 * i;
            const uint2 x = lds64(vd + row * St::kRow + 16 * v_chunk<D>(row, at >> 4) + (at & 8));
            d[0] = x.x;
            d[1] = x.y;
          }
        };
        load(x0, w[0]);
        load(x1, w[1]);
        load(y0, w[2]);
        load(y1, w[3]);
#pragma unroll
        for (int j = 0; j < (D == 64 ? 1 : 2); ++j) {   // 8 dimensions
          // bytes holding (first key's, second key's) codes of the even and odd dimensions
          constexpr uint32_t kLow = 0x0F0F0F0Fu;
          uint32_t ex[4], od[4], ey[4], oy[4];
          e2m1x8((w[0][j] & kLow) | ((w[1][j] << 4) & ~kLow), ex);
          e2m1x8(((w[0][j] >> 4) & kLow) | (w[1][j] & ~kLow), od);
          e2m1x8((w[2][j] & kLow) | ((w[3][j] << 4) & ~kLow), ey);
          e2m1x8(((w[2][j] >> 4) & kLow) | (w[3][j] & ~kLow), oy);
#pragma unroll
          for (int e = 0; e < 4; ++e) {          // dimensions 2 e and 2 e + 1 of the eight
            const uint32_t a0 = hmul2(ex[e], sx), a1 = hmul2(od[e], sx), a2 = hmul2(ey[e], sy), a3 = hmul2(oy[e], sy);
            const int t = (D == 64 ? 0 : 8 * i + 4 * j) + e;
#pragma unroll
            for (int nt = 0; nt < kRowTiles; ++nt) mma_f16(o[t][nt], a0, a1, a2, a3, p[mt][nt][0], p[mt][nt][1]);
          }
        }
      }
    }
  }
  if (bad_index) report(a.status, KVQ_STATUS_BAD_INDEX);

  // ---- join the four warps -------------------------------------------------
  const float v_scale = load_global(a.v_scale);        // under way meanwhile
  cp_wait<0>();
  __syncthreads();                               // every ring is idle
  float* jo = reinterpret_cast<float*>(smem);    // [kWarps][kRows][D]
  __shared__ float jm[kWarps][kRows], jl[kWarps][kRows];
#pragma unroll
  for (int nt = 0; nt < kRowTiles; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float sum = l[nt][x];
      sum += __shfl_xor_sync(kFull, sum, 4);
      sum += __shfl_xor_sync(kFull, sum, 8);
      sum += __shfl_xor_sync(kFull, sum, 16);
      const int r = 8 * nt + 2 * c + x;
      if (g == 0) {
        jm[warp][r] = m[nt][x];
        jl[warp][r] = sum;
      }
      // dimensions [g D/8, +D/8): two per tile
      float* dst = jo + (warp * kRows + r) * D + g * (D / 8);
#pragma unroll
      for (int t = 0; t < kDimTiles; ++t)
        *reinterpret_cast<float2*>(dst + 2 * t) = make_float2(o[t][nt][x], o[t][nt][2 + x]);
    }
  __syncthreads();
  __shared__ float cm[kRows], cl[kRows];         // of the four warps together, for the cluster
  for (int i = threadIdx.x; i < rows * (D / 8); i += kThreads) {
    const int r = i / (D / 8), d = (i % (D / 8)) * 8;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, jm[w][r]);
    float sum = 0.0f, acc[8] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      // a warp that saw nothing holds zeros
      const float f = jm[w][r] == -INFINITY ? 1.0f : ex2(jm[w][r] - top);
      sum += f * jl[w][r];
      const float4* src = reinterpret_cast<const float4*>(jo + (w * kRows + r) * D + d);
      const float4 u = src[0], v = src[1];
      acc[0] += f * u.x; acc[1] += f * u.y; acc[2] += f * u.z; acc[3] += f * u.w;
      acc[4] += f * v.x; acc[5] += f * v.y; acc[6] += f * v.z; acc[7] += f * v.w;
    }
    if (a.cluster) {                             // in the place of the first warp's, read by this thread only
      float4* dst = reinterpret_cast<float4*>(jo + r * D + d);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (d == 0) {
        cm[r] = top;
        cl[r] = sum;
      }
      continue;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float lse2 = sum == 0.0f ? -INFINITY : top + (log2f(sum) - kShift);
    const RowAt at = row_at(a, rq, head, static_cast<uint32_t>(row0 + r));
    if (a.num_splits > 1) {
      const int64_t pr = (at.token * a.num_heads + at.head) * a.num_splits + split;
      float4* dst = reinterpret_cast<float4*>(a.part_o + pr * D + d);
      dst[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
      dst[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
      if (d == 0) a.part_lse[pr] = lse2;
    } else {
      const float f = inv * v_scale;
      st16(static_cast<__nv_bfloat16*>(a.out) + at.token * a.out_stride_t + at.head * a.out_stride_h + d,
           make_uint4(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f),
                      pack_bf16x2(acc[4] * f, acc[5] * f), pack_bf16x2(acc[6] * f, acc[7] * f)));
      if (d == 0 && a.lse != nullptr) a.lse[at.token * a.lse_stride_t + at.head] = lse2 * kLn2;
    }
  }
  if (a.cluster)
    join_cluster(a, rq, head, row0, rows, split, D, smem_u32(jo), 4 * D, smem_u32(cm), smem_u32(cl));
}

// Joins the ranges of every row: with L_s the base-2 log-sum-exp of range s
// and o_s its normalised output, out = sum 2^(L_s - M) o_s / sum 2^(L_s - M).
// One warp per (token, head) row of a live request; a range that saw nothing
// (-inf) weighs nothing.  Latency bounds it, so the chain is short: the first
// ranges' rows are loaded beside their L_s, not after.  The call's own arrays
// are read after the wait like everything else: what an earlier kernel wrote
// is promised to be visible only there.
constexpr int kJoinWarps = 4;

template <int D, int kBatch>                             // kBatch: ranges in flight
__global__ void __launch_bounds__(kJoinWarps * 32, 4) per_head_join_kernel(const PerHeadAttentionArgs a) {
  const int64_t flat = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  wait_for_previous();
  const float v_scale = load_global(a.v_scale);          // in flight beside the request
  Request rq;
  if (!request_of(a, b, rq) || flat >= static_cast<int64_t>(rq.tokens) * a.num_heads) return;
  const int64_t row = rq.token0 * a.num_heads + flat;
  const float* ls = a.part_lse + row * a.num_splits;
  constexpr int kDims = D / 32;                          // per lane
  const float* po = a.part_o + row * a.num_splits * D + kDims * lane;
  float2 v[kBatch][kDims / 2];
  auto load = [&](int s0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int i = 0; i < kDims / 2; ++i)
        v[k][i] = s0 + k < a.num_splits ? *reinterpret_cast<const float2*>(po + static_cast<int64_t>(s0 + k) * D + 2 * i)
                                        : make_float2(0.0f, 0.0f);
  };
  // lane l holds ranges l, l + 32, ...
  constexpr int kPer = KVQ_PER_HEAD_MAX_SPLITS / 32;
  float own[kPer], top = -INFINITY;
  bool abandoned = false;
#pragma unroll
  for (int j = 0; j < kPer; ++j) own[j] = 32 * j + lane < a.num_splits ? ls[32 * j + lane] : -INFINITY;
  load(0);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    top = fmaxf(top, own[j]);
    abandoned |= __float_as_uint(own[j]) == kAbandoned;
  }
  if (__any_sync(kFull, abandoned)) return;              // a range whose CTA gave up: the row stays unwritten
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  float acc[kDims], den = 0.0f;
#pragma unroll
  for (int i = 0; i < kDims; ++i) acc[i] = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    own[j] = own[j] == -INFINITY ? 0.0f : ex2(own[j] - top);   // the range's weight
    den += own[j];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kFull, den, o);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    for (int s0 = 0; s0 < 32 && 32 * j + s0 < a.num_splits; s0 += kBatch) {
      if (j + s0 > 0) load(32 * j + s0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = __shfl_sync(kFull, own[j], s0 + k);
        // the row of an empty range was never written: what was loaded is not used
#pragma unroll
        for (int i = 0; i < kDims / 2; ++i) {
          acc[2 * i] += w == 0.0f ? 0.0f : w * v[k][i].x;
          acc[2 * i + 1] += w == 0.0f ? 0.0f : w * v[k][i].y;
        }
      }
    }
  }
  const float f = (den == 0.0f ? 0.0f : 1.0f / den) * v_scale;
  const int64_t token = row / a.num_heads, h = row - token * a.num_heads;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + token * a.out_stride_t +
                                              h * a.out_stride_h + kDims * lane);
#pragma unroll
  for (int i = 0; i < kDims; i += 2) dst[i / 2] = pack_bf16x2(acc[i] * f, acc[i + 1] * f);
  if (lane == 0 && a.lse != nullptr) a.lse[token * a.lse_stride_t + h] = den == 0.0f ? -INFINITY : (top + log2f(den)) * kLn2;
}

template <int D, int kRowTiles>
cudaError_t launch_rows(const PerHeadAttentionArgs& a, cudaStream_t stream) {
  constexpr int kSmem = kWarps * kStages * Stage<D>::kBytes;
  static_assert(kSmem >= kWarps * 8 * kRowTiles * D * 4, "the joined rows fit the rings");
  const cudaError_t e = cudaFuncSetAttribute(per_head_attention_kernel<D, kRowTiles>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(a.max_query_len) * a.group;
  const int64_t blocks = (rows + 8 * kRowTiles - 1) / (8 * kRowTiles);
  const dim3 grid(static_cast<unsigned>(blocks * a.num_kv_heads * a.num_splits), static_cast<unsigned>(a.batch_size));
  return launch_dependent(per_head_attention_kernel<D, kRowTiles>, grid, kThreads, kSmem, a.cluster ? a.num_splits : 1,
                          stream, a, static_cast<int32_t>(blocks));
}

template <int D>
cudaError_t launch_join(const PerHeadAttentionArgs& a, cudaStream_t stream) {
  const int64_t join = static_cast<int64_t>(a.max_query_len) * a.num_heads;
  const dim3 grid(static_cast<unsigned>((join + kJoinWarps - 1) / kJoinWarps), static_cast<unsigned>(a.batch_size));
  // as many ranges in flight as a row has, up to 16 (one user's tree in 16
  // ranges: 16.3 us, eight in flight 17.0), but no more: they cost registers,
  // and calls of few ranges have many rows (trees 32 x 64 in 4: 500 us, 523)
  return launch_dependent(a.num_splits <= 4 ? per_head_join_kernel<D, 4> : per_head_join_kernel<D, D == 256 ? 8 : 16>, grid,
                          kJoinWarps * 32, 0, 1, stream, a);
}

}  // namespace

cudaError_t launch_per_head_attention(const PerHeadAttentionArgs& a, int sms, cudaStream_t stream) {
  const int64_t block = per_head_block(static_cast<int64_t>(a.max_query_len) * a.group,
                                       static_cast<int64_t>(a.num_kv_heads) * a.batch_size, a.head_size, a.num_splits,
                                       a.cluster, sms);
  cudaError_t e;
  if (block > 16)
    e = launch_per_head_prefill(a, stream);
  else if (a.head_size == 64)
    e = block == 8 ? launch_rows<64, 1>(a, stream) : launch_rows<64, 2>(a, stream);
  else if (a.head_size == 128)
    e = block == 8 ? launch_rows<128, 1>(a, stream) : launch_rows<128, 2>(a, stream);
  else
    e = launch_rows<256, 1>(a, stream);
  if (e != cudaSuccess || a.num_splits == 1 || a.cluster) return e;
  return a.head_size == 64 ? launch_join<64>(a, stream)
                           : a.head_size == 128 ? launch_join<128>(a, stream) : launch_join<256>(a, stream);
}

}  // namespace kvq
