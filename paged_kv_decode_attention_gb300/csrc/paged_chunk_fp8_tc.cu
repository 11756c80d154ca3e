// paged_chunk_fp8_tc.cu -- attention of several query positions per request
// over a paged cache of E4M3 codes with a scale for each block and KV head,
// both contractions on the tensor cores' 8-bit path: a causal chunk behind
// cached tokens ("Chapter 8: Inference Optimization", clxhxhhr.top/posts/4341,
// §8.2.3), or a chain of drafted tokens (§8.5.2), with K and V in FP8 (§8.4.4).
//
// Mathematics.  Softmax over the visible keys, tile by tile (64 keys) with a
// running maximum and sum in FP32.  With value = code * scale, ks and vs the
// scales of a key's block:
//   S_ij = sum_d (sigma_i q_id) kcode_jd      (tensor cores, codes as they are)
//   y_ij = S_ij (scale / sigma_i) ks_j + log2(vs_j), in base 2
//   w_ij = 2^(y_ij - m_i), m_i a running maximum of y less a constant: so that
//          the weights are what the second product needs, in the range of their
//          type whatever vs is
//   O_i  = sum_j w_ij vcode_j,   l_i = sum_j w_ij / vs_j,   out = O_i / l_i
// Scales are constant over 16 keys, so they cost a few FP32 operations per 16
// scores.  8-bit products want both operands in 8 bits.  Queries enter S as two
// E4M3 parts (sigma_i a power of two that brings the row's largest magnitude
// to 2^7 .. 2^8: exact down to 2^-17 of it), against K's codes as they are: two
// products at twice the BF16 rate.
//
// kWide : 256 rows (64 positions x 4 heads) share a CTA's tiles, 128 a row
//         tile; while one row tile's softmax runs, the tensor cores work on
//         the other's products.  What bounds it is the softmax's arithmetic,
//         so the weights enter as one FP16 value (2^-11 relative) and four
//         warps convert each V tile to FP16, once for all rows.  (With two
//         E4M3 parts of each weight the softmax of a tile took 900 cycles of
//         a warp for its exponentials and parts, now as many as a prompt's.)
//         They enter times 2^7, so that FP16's range, 2^-24 .. 2^15, reaches
//         down to 2^-31 of the largest.
// !kWide: up to kRows rows, 32, 64 or 128.  HBM is the bound, and a chain of
//         scores, softmax and product is longer than a tile's transfer.  So
//         the CTA's two halves take the even and the odd tiles of keys, and
//         where there are few query rows they are laid out twice: a copy's
//         threads do the softmax of half of a tile's keys, with a maximum and a
//         sum of their own (the other keys' weights are zeros).  At the end
//         all copies and both halves are joined through shared memory.  Up to
//         32 rows the products have M = 64, which reads half as much of the
//         queries per product, and two threads share a row.  V's codes enter
//         as they are and the weights as three E5M2 parts times 2^13, by way
//         of FP16 (2^-8 relative, down to 2^-30 of the largest).  (With two
//         E4M3 parts, which lose what lies below 2^-16 of the largest, and
//         two buffers for them, 37 x 7 took 38 us, not 43: half of the
//         difference is the third part's two products.)
//
// Scores (64 columns), the weights (32, their parts 48) and O lie in a row
// tile's 256 columns of tensor memory.  The next scores are issued as soon as the
// softmax holds the present ones in registers, ahead of the product that waits
// for their weights: neither side waits for the other's latency.
//
// Measured, 32 query and 8 KV heads: 4 x 2000 queries behind 4000 to 8000
// tokens 0.79 ms, 1.3 PFLOP/s (tiles of 128 keys with scores and weights in one
// buffer, one chain: 1.09); 37 x 7 behind 2048 to 2303 43 us, 4.0 TB/s (57): the
// products' issue, the start, 6000 cycles to the first scores, the ends of jobs,
// 3,500 each, and the joining kernel.  37 requests behind 2100 tokens, by the
// rows' layout: 8 queries 42 us with M = 64, 50 with 64 rows of M = 128, 62 with
// 128; 16 queries 55 with 64 rows, 67 with 128, 67 as kWide; 24 queries 70 with
// 128, 74 as kWide; 32 queries 74 with 128, 78 as kWide.
//
// Work is cut by tiles, not by requests (pkv_shares.cuh); a cut job leaves
// un-normalised FP32 partials.
//
// CTA = 16 warps:
//   warps 0-7: softmax, one thread per row (TMEM lane), a warpgroup per row
//             tile (or half of the tiles).
//   warp 8  : TMA producer of K (kWide: and V): 16-token boxes of 2 KiB, 128-byte
//             swizzle; blocks past the range arrive as zeros.  A box takes some
//             70 cycles to issue.
//   warps 9, 10: MMA issuers, one per row tile (or half).
//   warp 11 : finds the CTA's pieces and fetches the blocks' scales.
//   warps 12-15: the query operand, a piece ahead; kWide: V to FP16; !kWide: warp
//             12 is V's producer instead.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstddef>

#include "pkv_common.cuh"
#include "pkv_kernels.h"
#include "pkv_shares.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kCfTokens = 64;                         // keys of a tile
constexpr int kCfTileBlocks = kCfTokens / kBlockSize;  // 4
constexpr int kCfTileBytes = kCfTokens * kHeadDim;    // K or V of a tile: 8 KiB
constexpr int kCfBoxBytes = kBlockSize * kHeadDim;
constexpr int kCfGroupTiles = 32 / kCfTileBlocks;     // tiles whose blocks a warp looks up at a time
constexpr int kCfScaleGroups = 2;                     // groups whose scales are held
constexpr int kCfThreads = 512;
constexpr int kCfRows = 128;
constexpr int kCfPos = kCfRows / kGroup;              // positions of a row tile
constexpr int kCfPartBytes = kCfRows * kHeadDim;      // one part of a row tile's queries: 16 KiB
constexpr int kCfV16Bytes = 2 * kCfTileBytes;         // a V tile in FP16, two 64-dim halves
constexpr int kCfV16Stages = 3;
constexpr int kCfScaleFloats = 3 * kCfTileBlocks;     // ks, log2 vs, 1 / vs
constexpr int kCfHelpers = 4;                         // warps 12-15

template <bool kWide>
struct CfShape {
  static constexpr int kSlots = kWide ? 14 : 16;      // ring: K, V, K, V, ...
  // queries, [row tile] or [buffer], each [high, low parts]
  static constexpr int kOffQ = 0;
  static constexpr int kOffExtra = 4 * kCfPartBytes;  // V in FP16, or the join's buffer, FP32 [2 x 128][32]
  static constexpr int kOffRing = kOffExtra + (kWide ? kCfV16Stages * kCfV16Bytes : 2 * kCfRows * 32 * 4);
  static constexpr int kOffScale = kOffRing + kSlots * kCfTileBytes;
  static constexpr int kOffSigma = kOffScale + kCfScaleGroups * kCfGroupTiles * kCfScaleFloats * 4;  // FP32 [2][128]: scale / sigma
  static constexpr int kOffBar = kOffSigma + 2 * kCfRows * 4;
  static constexpr int kSmem = kOffBar + 896;
  static_assert(kSmem <= 227 * 1024, "one CTA per SM");
  static_assert(kOffBar % 16 == 0 && kOffScale % 16 == 0 && kOffRing % 1024 == 0, "alignment");
};

constexpr uint32_t kCfTileCols = 256;                 // S, weights, O
constexpr uint32_t kCfColP = 64;
constexpr uint32_t kCfPartCols = 16;                  // !kWide: a part of the weights
constexpr uint32_t kCfColO = 128;
constexpr uint32_t kCfColQ = 96;                      // kWide: the queries' high parts, behind the weights
constexpr int kCfSoftmaxRegs = 168;
constexpr int kCfOtherRegs = 88;
static_assert((2 * kCfSoftmaxRegs + 2 * kCfOtherRegs) * 128 <= 128 * kCfThreads, "register split");
// Base 2: weights stay at or below 2^15 (E5M2 reaches 1.75 times that, FP16
// twice).  A new maximum is given 2^13, or 2^7, and room to be exceeded.
constexpr float kCfTop = 15.f;
constexpr float cf_start(bool wide) { return wide ? 7.f : 13.f; }
// The queries' parts are cut from FP16 values 2^-8 of what they stand for.
constexpr float kCfCodeUnit = 256.f;
// Least factor of a score: below it scores are as good as zero, and a product
// of scales that vanishes would turn masked ones, -inf, into NaN.
constexpr float kCfLeast = 0x1p-100f;
// In tiles: what a job costs besides its tiles, and the least worth a CTA.
constexpr int kCfJobCost = 8;
constexpr int kCfMinShare = 12;

struct alignas(16) CfPiece {
  int32_t r, rt, kvh;   // request, row tile (pair), KV head
  int32_t begin, take;  // tiles [begin, begin + take)
  int32_t n;            // of n; 0: no more pieces
  int32_t pad0, pad1;
};

template <bool kWide>
struct CfBars {
  uint64_t full[CfShape<kWide>::kSlots], empty[CfShape<kWide>::kSlots];
  uint64_t sc_full[kCfScaleGroups], sc_empty[kCfScaleGroups];
  uint64_t q_full[2], q_empty[2];  // per row tile, or buffer
  uint64_t qt_full[2];             // kWide: the high parts are in tensor memory
  uint64_t v16_full[kCfV16Stages], v16_empty[kCfV16Stages];
  uint64_t join_full, join_free;   // !kWide: the join's buffer is written, is read
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2][2];
  uint64_t o_done[2][2];           // (two: nobody waits for each of them in turn)
  uint64_t u_full[2], u_empty[2];
  CfPiece piece[2];
  uint32_t tmem_base;
};
static_assert(sizeof(CfBars<true>) <= 896 && offsetof(CfBars<true>, piece) % 16 == 0, "barrier area");
static_assert(sizeof(CfBars<false>) <= 896 && offsetof(CfBars<false>, piece) % 16 == 0, "barrier area");

template <int kRegs>
__device__ __forceinline__ void cf_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void cf_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// D[tmem] (+)= A[tmem] * B[smem], 8-bit floating-point operands (A: four to a column).
__device__ __forceinline__ void mma_f8_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 4 weights as the bytes of their three E5M2 parts.
__device__ __forceinline__ void cf_weights(float p0, float p1, float p2, float p3, uint32_t& hi, uint32_t& mid,
                                           uint32_t& lo) {
  uint32_t h0, h1, m0, m1, l0, l1;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h0) : "f"(p1), "f"(p0));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h1) : "f"(p3), "f"(p2));
  tc::e5m2_parts(h0, m0, l0);
  tc::e5m2_parts(h1, m1, l1);
  hi = __byte_perm(h0, h1, 0x7531);
  mid = __byte_perm(m0, m1, 0x7531);
  lo = __byte_perm(l0, l1, 0x7531);
}

// 4 signed values (2^-8 of what the parts stand for) as the bytes of their high
// parts, E4M3 cut to 4 significant bits, and of what that leaves, rounded to 4.
// (FP16's exponent field is E4M3's here, subnormals included, so both parts
// come by masks and shifts.)
__device__ __forceinline__ void cf_signed(float x0, float x1, float x2, float x3, uint32_t& hi, uint32_t& lo) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h0) : "f"(x1), "f"(x0));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h1) : "f"(x3), "f"(x2));
  const uint32_t a0 = h0 & 0x7fff7fffu, a1 = h1 & 0x7fff7fffu;
  uint32_t r0, r1;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r0) : "r"(a0), "r"(a0 & 0xff80ff80u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(a1), "r"(a1 & 0xff80ff80u));
  uint32_t sign;  // each value's sign over its byte
  asm("prmt.b32 %0, %1, %2, 0xfdb9;" : "=r"(sign) : "r"(h0), "r"(h1));
  sign &= 0x80808080u;
  hi = __byte_perm(a0 << 1, a1 << 1, 0x7531) | sign;
  lo = __byte_perm(r0 * 2 + 0x00800080u, r1 * 2 + 0x00800080u, 0x7531) | sign;
}

// sigma, the power of two that brings a row's largest |q| (BF16 bits) into
// [2^7, 2^8), over the parts' unit, 2^8; `inv` = 1 / sigma.  1 for zeros; NaN for
// infinities and NaN, so that all the row's parts and scores are NaN (an
// infinity's bits would be those of a finite code).
__device__ __forceinline__ float cf_sigma(uint32_t amax_bits, float& inv) {
  const int e = amax_bits == 0 ? 7 : max(static_cast<int>(amax_bits >> 7) - 127, -113);  // (subnormals: as 2^-113)
  inv = __int_as_float((127 + e - 7) << 23);
  return amax_bits >= 0x7f80u ? NAN : __int_as_float((127 + 7 - e) << 23) * (1.f / kCfCodeUnit);
}

// 16 E4M3 codes as FP16 (exact).
__device__ __forceinline__ void cf_to_half(const uint4& c, uint4& a, uint4& b) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint16_t pair = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[i]) : "h"(pair));
  }
  a = make_uint4(h[0], h[1], h[2], h[3]);
  b = make_uint4(h[4], h[5], h[6], h[7]);
}

__device__ __forceinline__ uint32_t cf_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Tiles of keys that a row tile of a request reads.
__device__ __forceinline__ int cf_tiles(const ScaledArgs& a, int pair, int n_rt, int pos) {
  const int r = n_rt == 1 ? pair : pair / n_rt;
  const int rt = pair - r * n_rt;
  const int ctx = min(max(a.context_lens[r], 0), a.max_blocks * kBlockSize);
  const int end = ctx - max(a.q_len - (rt + 1) * pos, 0);
  return end > 0 ? (end + kCfTokens - 1) / kCfTokens : 0;
}

// How the query rows of a call lie in the products and the threads.
template <bool kWide, int kRows>
struct CfRowsOf {
  static constexpr bool kHalf = !kWide && kRows == 32;           // M = 64: 16 rows and two threads a row in a warp
  static constexpr int kMma = kHalf ? 64 : kCfRows;              // M
  static constexpr int kWarpRows = kHalf ? 16 : 32;
  static constexpr int kCopies = kMma / kRows;
  static constexpr int kCopyKeys = kCfTokens / kCopies;          // of a tile's keys
  static constexpr int kCols = kHalf ? kCopyKeys / 2 : kCopyKeys;  // a thread's
};

template <bool kWide, int kRows>
__global__ void __launch_bounds__(kCfThreads, 1)
    paged_chunk_fp8_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                              const ScaledArgs a) {
  using S = CfShape<kWide>;
  using R = CfRowsOf<kWide, kRows>;
  constexpr uint32_t kSlots = S::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  auto* bars = reinterpret_cast<CfBars<kWide>*>(smem + S::kOffBar);
  auto uniform = [](int x) -> int { return __shfl_sync(0xffffffffu, x, 0); };
  const int warp = uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  constexpr int kQWarps = kWide ? kCfHelpers : kCfHelpers - 1;  // that write the query operand

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < kSlots; ++s) {
      mbar_init(&bars->full[s], 1);
      // K (even places): both issuers, or the half's; V: the converting warps, or the half's
      mbar_init(&bars->empty[s], kWide ? ((s & 1) ? kCfHelpers : 2) : 1);
    }
    for (int s = 0; s < kCfScaleGroups; ++s) {
      mbar_init(&bars->sc_full[s], 1);
      mbar_init(&bars->sc_empty[s], 8);  // the softmax warps
    }
    for (int s = 0; s < kCfV16Stages; ++s) {
      mbar_init(&bars->v16_full[s], kCfHelpers);
      mbar_init(&bars->v16_empty[s], 2);
    }
    mbar_init(&bars->join_full, 256);
    mbar_init(&bars->join_free, 256);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], kQWarps);
      mbar_init(&bars->q_empty[t], kWide ? 5 : 10);  // the softmax warps and issuers that use it
      mbar_init(&bars->qt_full[t], 128);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->s_free[t], 128);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->p_full[t][b], 128);
        mbar_init(&bars->o_done[t][b], 1);
      }
      mbar_init(&bars->u_full[t], 1);
      mbar_init(&bars->u_empty[t], 15);  // every other warp
    }
    fence_barrier_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tc::prefetch_tensor_map(&k_map);
    tc::prefetch_tensor_map(&v_map);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_wait();  // everything below may read what earlier grids in the stream write
  pdl_trigger();

  constexpr int kPos = kWide ? 2 * kCfPos : kCfPos;  // positions of a piece
  const int n_rt = kWide ? (a.q_len + kPos - 1) / kPos : 1;
  const int pairs = a.num_seqs * n_rt;
  const int hq = a.num_kv_heads * kGroup;
  const uint32_t tmem = uniform(bars->tmem_base);
  const uint32_t sbase = uniform(smem_addr(smem));
  bool ok = true;

  uint32_t walked = 0;
  auto next_piece = [&](CfPiece& u) -> bool {
    const int slot = walked & 1;
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->u_full[slot], (walked >> 1) & 1));
    if (!ok) return false;
    const int4 x = reinterpret_cast<const int4*>(&bars->piece[slot])[0];
    const int4 y = reinterpret_cast<const int4*>(&bars->piece[slot])[1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->u_empty[slot]);
    ++walked;
    u.r = uniform(x.x);
    u.rt = uniform(x.y);
    u.kvh = uniform(x.z);
    u.begin = uniform(x.w);
    u.take = uniform(y.x);
    u.n = uniform(y.y);
    return u.n > 0;
  };
  // The query buffer of the k-th piece for row tile t, and its phase there.
  auto q_slot = [](uint32_t k, int t) -> uint32_t { return kWide ? t : k & 1; };
  auto q_phase = [](uint32_t k) -> uint32_t { return kWide ? k & 1 : (k >> 1) & 1; };
  // tiles of the piece that half t works on
  auto tiles_of = [&](const CfPiece& u, int t) -> int { return kWide ? u.take : (u.take - t + 1) >> 1; };

  if (warp >= 8) {
    cf_regs_down<kCfOtherRegs>();
    if (warp == 11) {
      // ------------------------ pieces and scales ------------------------
      const Share share = find_share(pairs, a.num_kv_heads, kCfJobCost, kCfMinShare, lane,
                                     [&](int p) -> int { return cf_tiles(a, p, n_rt, kPos); });
      int pair = share.row, kvh = share.kvh, n = share.tiles, into = share.into, left = share.left;
      auto place = [&](int& r, int& rt) {  // of the pair
        r = n_rt == 1 ? pair : pair / n_rt;
        rt = pair - r * n_rt;
      };
      if (lane == 0) {  // for the joining kernel
        CfCut cut{};
        place(cut.r, cut.rt);
        cut.kvh = kvh;
        cut.n = n;
        cut.into = into;
        cut.per = share.per;
        a.cuts[blockIdx.x] = cut;
      }
      uint32_t sets = 0;  // groups of scales written so far
      // the scales of a piece's blocks, 32 blocks (8 tiles) at a time, fetched a group ahead
      auto scales_of = [&](const CfPiece& u) {
        const int32_t* table = a.block_tables + static_cast<int64_t>(u.r) * a.max_blocks;
        const int ctx = min(max(a.context_lens[u.r], 0), a.max_blocks * kBlockSize);
        const int last = (ctx + kBlockSize - 1) / kBlockSize;  // blocks past the context have no scale
        auto fetch = [&](int group, float& ks, float& vs) {
          const int lb = (u.begin + kCfGroupTiles * group) * kCfTileBlocks + lane;
          ks = vs = 1.f;
          if (lb < last && lb < (u.begin + u.take) * kCfTileBlocks) {
            int b = table[lb];
            if (b < 0 || b >= a.num_blocks) b = 0;  // (reported by the producer)
            const int64_t at = static_cast<int64_t>(b) * a.num_kv_heads + u.kvh;
            ks = a.k_scales[at];
            vs = a.v_scales[at];
          }
        };
        const int groups = (u.take + kCfGroupTiles - 1) / kCfGroupTiles;
        float ks, vs, ks_next = 1.f, vs_next = 1.f;
        fetch(0, ks, vs);
        for (int g = 0; g < groups && ok; ++g) {
          if (g + 1 < groups) fetch(g + 1, ks_next, vs_next);
          const int slot = sets % kCfScaleGroups;
          if (sets >= kCfScaleGroups)
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->sc_empty[slot], ((sets / kCfScaleGroups) & 1) ^ 1));
          if (!ok) break;
          float* dst = reinterpret_cast<float*>(smem + S::kOffScale) +
                       (slot * kCfGroupTiles + lane / kCfTileBlocks) * kCfScaleFloats + lane % kCfTileBlocks;
          dst[0] = ks;
          dst[kCfTileBlocks] = log2f(vs);
          dst[2 * kCfTileBlocks] = 1.f / vs;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->sc_full[slot]);
          ++sets;
          ks = ks_next;
          vs = vs_next;
        }
      };
      CfPiece now{}, was{};
      for (uint32_t round = 0;; ++round) {
        was = now;
        now = CfPiece{};
        while (left > 0 && now.n == 0) {
          int begin, take;
          take_of_job(n, kCfJobCost, into, left, begin, take);
          if (take > 0) {
            place(now.r, now.rt);
            now.kvh = kvh;
            now.begin = begin;
            now.take = take;
            now.n = n;
          }
          if (++kvh == a.num_kv_heads) {  // (the next job starts here, if anything is left)
            kvh = 0;
            for (++pair; left > 0 && pair < pairs && (n = cf_tiles(a, pair, n_rt, kPos)) == 0; ++pair) {
            }
          }
        }
        const int slot = round & 1;
        if (round >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&bars->u_empty[slot], ((round >> 1) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          bars->piece[slot] = now;
          mbar_arrive(&bars->u_full[slot]);
        }
        __syncwarp();
        if (round > 0) scales_of(was);
        if (!ok || now.n == 0) break;
      }
      if (!ok && lane == 0) report(a.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 8 || (!kWide && warp == 12)) {
      // ---------------------------- TMA producers ----------------------------
      // kWide: K of a tile in lanes 0-3, V in lanes 4-7.
      // read once, unless several row tiles of the request read the same blocks
      const uint64_t policy = n_rt > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
      const int oob_row = a.num_blocks * a.num_kv_heads * kBlockSize;  // first row past the pool
      const bool is_v = kWide ? lane >= kCfTileBlocks : warp == 12;
      constexpr int kLanes = kWide ? 2 * kCfTileBlocks : kCfTileBlocks;
      uint32_t filled = 0;  // tiles so far
      CfPiece u;
      while (next_piece(u)) {
        const int32_t* table = a.block_tables + static_cast<int64_t>(u.r) * a.max_blocks;
        const int ctx = min(max(a.context_lens[u.r], 0), a.max_blocks * kBlockSize);
        const int last = (ctx + kBlockSize - 1) / kBlockSize;
        const int b0 = u.begin * kCfTileBlocks, b1 = min(last, b0 + u.take * kCfTileBlocks);
        auto row_of = [&](int i, int id) -> int {  // pool row of the piece's i-th block
          if (b0 + i >= b1) return oob_row;
          if (id < 0 || id >= a.num_blocks) {
            report(a.err, PKV_DEVERR_BLOCK_ID);
            id = 0;
          }
          return (id * a.num_kv_heads + u.kvh) * kBlockSize;
        };
        auto entry = [&](int i) -> int { return table[min(b0 + i, a.max_blocks - 1)]; };
        int cur = row_of(lane, entry(lane)), next = 0;
        for (int j = 0; j < u.take && ok; ++j, ++filled) {
          const int in_group = j % kCfGroupTiles;
          if (in_group == 0) next = entry(kCfTileBlocks * j + 32 + lane);  // the next tiles' ids
          const int y = __shfl_sync(0xffffffffu, cur, in_group * kCfTileBlocks + lane % kCfTileBlocks);
          if (in_group == kCfGroupTiles - 1) cur = row_of(kCfTileBlocks * (j + 1) + lane, next);
          const uint32_t place = 2 * filled + (is_v ? 1 : 0);
          const uint32_t slot = place % kSlots;
          bool mine = true;
          if (place >= kSlots) mine = mbar_wait(&bars->empty[slot], ((place / kSlots) & 1) ^ 1);
          ok = __all_sync(0xffffffffu, mine);
          if (!ok) break;
          if (lane < kLanes && lane % kCfTileBlocks == 0) mbar_arrive_expect_tx(&bars->full[slot], kCfTileBytes);
          __syncwarp();
          if (lane < kLanes)
            tc::tma_load_2d(smem + S::kOffRing + slot * kCfTileBytes + lane % kCfTileBlocks * kCfBoxBytes,
                            is_v ? &v_map : &k_map, 0, y, &bars->full[slot], policy);
        }
        if (!ok) break;
      }
      if (lane < kLanes && lane % kCfTileBlocks == 0 && !ok) {
        report(a.err, PKV_DEVERR_TIMEOUT);
        // copies under way must land before shared memory is released
        for (uint32_t f = filled > kSlots / 2 ? filled - kSlots / 2 : 0; f < filled; ++f) {
          const uint32_t place = 2 * f + (is_v ? 1 : 0);
          mbar_wait(&bars->full[place % kSlots], (place / kSlots) & 1);
        }
      }
      __syncwarp();
    } else if (warp >= 12) {
      // ---------------- the query operand; kWide: V to FP16 ----------------
      const int who = warp - (16 - kQWarps);
      const int c16 = lane & 7;  // 8 lanes a row, 16 dims each
      // the queries of piece u (its number in the walk: k), 4 rows an iteration
      auto queries = [&](const CfPiece& u, uint32_t k) {
        for (int t = 0; t < (kWide ? 2 : 1) && ok; ++t) {
          const uint32_t buf = q_slot(k, t);
          const uint32_t uses = kWide ? k : k >> 1;  // of the buffer before
          if (uses > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_empty[buf], (uses & 1) ^ 1));
          if (!ok) break;
          const int pos0 = u.rt * kPos + t * kCfPos;
          const int live_rows = max(min(pos0 + kCfPos, a.q_len) - pos0, 0) * kGroup;
          uint8_t* qa = smem + S::kOffQ + buf * 2 * kCfPartBytes;
          float* inv_sigma = reinterpret_cast<float*>(smem + S::kOffSigma) + buf * kCfRows;
          constexpr int kIters = kRows / 4;
          for (int i0 = who; i0 < kIters && 4 * i0 < live_rows; i0 += 4 * kQWarps) {
            uint4 w[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int m = 4 * (i0 + i * kQWarps) + (lane >> 3);
              w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
              if (m < live_rows) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(a.q) +
                    ((static_cast<int64_t>(u.r) * a.q_len + pos0 + (m >> 2)) * hq + u.kvh * kGroup + (m & 3)) * kHeadDim +
                    16 * c16);
                w[i][0] = src[0];
                w[i][1] = src[1];
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int m = 4 * (i0 + i * kQWarps) + (lane >> 3);
              if (4 * (i0 + i * kQWarps) >= kRows) break;
              const uint32_t wv[8] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w,
                                      w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
              uint32_t top = wv[0] & 0x7fff7fffu;  // pairs of magnitudes: BF16 bits in the order of integers
#pragma unroll
              for (int e = 1; e < 8; ++e) top = __vmaxu2(top, wv[e] & 0x7fff7fffu);
#pragma unroll
              for (int off = 1; off < 8; off <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, off));
              float inv;
              const float f = cf_sigma(max(top & 0xffffu, top >> 16), inv);
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                cf_signed(bf16_lo(wv[2 * e]) * f, bf16_hi(wv[2 * e]) * f, bf16_lo(wv[2 * e + 1]) * f,
                          bf16_hi(wv[2 * e + 1]) * f, hi[e], lo[e]);
#pragma unroll
              for (int copy = 0; copy < R::kCopies; ++copy) {
                const uint32_t at = tc::sw128_offset_b8(m + copy * kRows, 16 * c16);
                *reinterpret_cast<uint4*>(qa + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(qa + kCfPartBytes + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (c16 == 0) inv_sigma[m + copy * kRows] = a.scale_log2 * inv;
              }
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->q_full[buf]);
        }
      };
      uint32_t k = 0;     // pieces so far
      uint32_t tile = 0;  // kWide: V tiles so far
      CfPiece u, after{};
      for (bool more = next_piece(u); more; u = after) {
        queries(u, k);
        ++k;
        more = next_piece(after);
        if constexpr (kWide) {
          if (more) {  // its queries towards L2: they are wanted in a hurry
            const int pos0 = after.rt * kPos;
            const uint16_t* q0 = static_cast<const uint16_t*>(a.q) +
                                 ((static_cast<int64_t>(after.r) * a.q_len + pos0) * hq + after.kvh * kGroup) * kHeadDim;
            const int lines = min(kPos, a.q_len - pos0) * (kGroup * kHeadDim * 2 / 128);
            for (int i = who * 32 + lane; i < lines; i += kCfHelpers * 32)
              prefetch_l2(q0 + static_cast<int64_t>(i >> 3) * hq * kHeadDim + (i & 7) * 64);
          }
          const int ctx = min(max(a.context_lens[u.r], 0), a.max_blocks * kBlockSize);
          for (int j = 0; j < u.take && ok; ++j, ++tile) {
            const uint32_t place = 2 * tile + 1, slot = place % kSlots, st = tile % kCfV16Stages;
            bool there = mbar_wait(&bars->full[slot], (place / kSlots) & 1);
            if (tile >= kCfV16Stages)
              there = there && mbar_wait(&bars->v16_empty[st], ((tile / kCfV16Stages) & 1) ^ 1);
            ok = __all_sync(0xffffffffu, there);
            if (!ok) break;
            const uint8_t* raw = smem + S::kOffRing + slot * kCfTileBytes;
            uint8_t* half = smem + S::kOffExtra + st * kCfV16Bytes;
            const int end = ctx - (u.begin + j) * kCfTokens;  // rows from here on hold nothing: zeros
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // 16 codes a lane, 4 rows a warp
              const int row = who * 16 + 4 * i + (lane >> 3);
              uint4 code = *reinterpret_cast<const uint4*>(raw + row * 128 + ((c16 ^ (row & 7)) << 4));
              if (row >= end) code = make_uint4(0, 0, 0, 0);
              uint4 h[2];
              cf_to_half(code, h[0], h[1]);
              // 64-dim half c16 / 4; the halves' lanes store in opposite order (banks)
              uint8_t* dst = half + (c16 >> 2) * kCfTileBytes + row * 128;
              const int o = c16 >> 2;
              const int ch = 2 * (c16 & 3);
              *reinterpret_cast<uint4*>(dst + (((ch + o) ^ (row & 7)) << 4)) = o ? h[1] : h[0];
              *reinterpret_cast<uint4*>(dst + (((ch + 1 - o) ^ (row & 7)) << 4)) = o ? h[0] : h[1];
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bars->empty[slot]);
              mbar_arrive(&bars->v16_full[st]);
            }
          }
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) report(a.err, PKV_DEVERR_TIMEOUT);
      __syncwarp();
    } else {
      // ---------------------------- MMA issuers ----------------------------
      constexpr uint32_t kIdS = tc::idesc_e4m3_f32(R::kMma, kCfTokens, false, false);
      constexpr uint32_t kIdO = kWide ? tc::idesc_f16_f32(kCfRows, kHeadDim, false, true)
                                      : tc::idesc_e4m3_f32(R::kMma, kHeadDim, false, true) | tc::kIdescE5m2A;
      const int t = warp - 9;
      const bool leader = lane == 0;
      const uint32_t scol = tmem + t * kCfTileCols;
      const uint64_t q_desc = tc::smem_desc(sbase + S::kOffQ, 16, 1024);
      const uint64_t ring = tc::smem_desc(sbase + S::kOffRing, 16, 1024);
      const uint64_t v16 = tc::smem_desc(sbase + S::kOffExtra, kCfTileBytes, 1024);
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity));
      };
      auto wait_full = [&](uint32_t place) -> bool { return wait(&bars->full[place % kSlots], (place / kSlots) & 1); };
      // two barriers, both tried before either result is looked at
      auto wait2 = [&](uint64_t* x, uint32_t xp, uint64_t* y, uint32_t yp) -> bool {
        const bool rx = mbar_try_wait(x, xp), ry = mbar_try_wait(y, yp);
        return __all_sync(0xffffffffu, (rx || mbar_wait(x, xp)) && (ry || mbar_wait(y, yp)));
      };
      // Stages go back by plain arrivals once a later wait has shown that the
      // products that read them are done.
      auto give_back = [&](uint32_t place) {
        if (leader) mbar_arrive(&bars->empty[place % kSlots]);
      };
      auto give_back_v = [&](uint32_t place, uint32_t tile) {  // (kWide: the converted tile)
        if (!kWide) {
          give_back(place);
        } else if (leader) {
          mbar_arrive(&bars->v16_empty[tile % kCfV16Stages]);
        }
      };
      // S = (high + low parts of the queries) K^T
      auto issue_s = [&](uint32_t place, uint32_t buf, bool last) {
        const uint64_t qd = q_desc + buf * (2 * kCfPartBytes >> 4);
        const uint64_t kd = ring + (place % kSlots) * (kCfTileBytes >> 4);
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (kWide && kk < 4)
              mma_f8_tmem_a(scol, scol + kCfColQ + 8 * kk, kd + ((32 * kk) >> 4), kIdS, kk > 0 ? 1u : 0u);
            else
              tc::mma_f8(scol, qd + (((kk >> 2) * kCfPartBytes + 32 * (kk & 3)) >> 4), kd + ((32 * (kk & 3)) >> 4), kIdS,
                       kk > 0 ? 1u : 0u);
          tc::commit(&bars->s_full[t]);
          if (last) tc::commit(&bars->q_empty[buf]);  // other queries may come
        }
        __syncwarp();
      };
      // O += P V: FP16, or (the three parts of the weights) V's codes
      auto issue_pv = [&](uint32_t place, uint32_t tile, uint32_t buf, bool first) {
        const uint64_t vd = kWide ? v16 + (tile % kCfV16Stages) * (kCfV16Bytes >> 4)
                                  : ring + (place % kSlots) * (kCfTileBytes >> 4);
        const uint32_t pcol = scol + kCfColP;
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < (kWide ? 4 : 6); ++kk) {
            if constexpr (kWide) {  // 16 keys
              tc::mma_bf16_tmem_a(scol + kCfColO, pcol + 8 * kk, vd + kk * (2048 >> 4), kIdO, (!first || kk > 0) ? 1u : 0u);
              continue;
            }
            const int slice = kk & 1;  // of 32 keys
            mma_f8_tmem_a(scol + kCfColO, pcol + kCfPartCols * (kk >> 1) + 8 * slice, vd + slice * (4096 >> 4), kIdO,
                          (!first || kk > 0) ? 1u : 0u);
          }
          tc::commit(&bars->o_done[t][buf]);
        }
        __syncwarp();
      };
      constexpr uint32_t kStep = kWide ? 2 : 4;  // ring places from one of its tiles to the next
      uint32_t c0 = 0;                           // ring place of the piece's first tile
      uint32_t g = 0;                            // tiles of this half so far
      uint32_t pieces = 0;
      CfPiece u;
      while (next_piece(u)) {
        const int n_t = tiles_of(u, t);
        uint32_t c = c0 + (kWide ? 0 : 2 * t);  // place of the present tile's K; its V is at c + 1
        c0 += 2 * u.take;
        const uint32_t qb = q_slot(pieces, t);
        ok = wait(&bars->q_full[qb], q_phase(pieces));
        if (kWide) ok = ok && wait(&bars->qt_full[t], pieces & 1);
        ++pieces;
        if (ok && n_t > 0) {
          ok = wait_full(c);
          if (ok) issue_s(c, qb, n_t == 1);
        }
        for (int j = 0; j < n_t && ok; ++j, ++g, c += kStep) {
          // The scores are in registers.  (They were committed after the
          // product of two tiles before, so that is done too.)
          const uint32_t ahead = c + kStep;
          ok = j + 1 < n_t ? wait2(&bars->full[ahead % kSlots], (ahead / kSlots) & 1, &bars->s_free[t], g & 1)
                           : wait(&bars->s_free[t], g & 1);
          if (!ok) break;
          give_back(c);
          if (j >= 2) give_back_v(c + 1 - 2 * kStep, g - 2);
          if (j + 1 < n_t) issue_s(ahead, qb, j + 2 == n_t);
          const uint32_t vp = c + 1;
          ok = kWide ? wait2(&bars->v16_full[g % kCfV16Stages], (g / kCfV16Stages) & 1, &bars->p_full[t][g & 1], (g >> 1) & 1)
                     : wait2(&bars->full[vp % kSlots], (vp / kSlots) & 1, &bars->p_full[t][g & 1], (g >> 1) & 1);
          if (!ok) break;
          issue_pv(vp, g, g & 1, j == 0);
        }
        // the last two tiles' V, once their products are done
        for (int back = min(n_t, 2); back > 0 && ok; --back) {
          ok = wait(&bars->o_done[t][(g - back) & 1], ((g - back) >> 1) & 1);
          if (ok) give_back_v(c + 1 - back * kStep, g - back);
        }
        if (!ok) break;
        if (n_t == 0 && leader) mbar_arrive(&bars->q_empty[qb]);
      }
      if (!ok && leader) report(a.err, PKV_DEVERR_TIMEOUT);
      __syncwarp();
    }
  } else {
    // ---------------------------- softmax ----------------------------
    cf_regs_up<kCfSoftmaxRegs>();
    const int t = warp >> 2;
    const int quad = warp & 3;  // TMEM sub-partition of this warp
    const uint32_t scol = tmem + (static_cast<uint32_t>(quad * 32) << 16) + t * kCfTileCols;
    const int row_tile = kWide ? t : 0;  // row tile of this warpgroup's rows

    if (blockIdx.x == 0)
      for (int r = threadIdx.x; r < a.num_seqs; r += 256)
        if (a.context_lens[r] > a.max_blocks * kBlockSize) report(a.err, PKV_DEVERR_CONTEXT);
    // rows that see no key at all belong to no piece: zeros
    for (int p = blockIdx.x; p < pairs; p += gridDim.x) {
      if (cf_tiles(a, p, n_rt, kPos) > 0) continue;
      const int64_t r = p / n_rt;
      const int pos0 = (p - static_cast<int>(r) * n_rt) * kPos;
      const int64_t chunks = static_cast<int64_t>(min(kPos, a.q_len - pos0)) * hq * (kHeadDim * 2 / 16);
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (r * a.q_len + pos0) * hq * kHeadDim);
      for (int64_t i = threadIdx.x; i < chunks; i += 256) o[i] = make_uint4(0, 0, 0, 0);
    }

    // this warp's copy of the query rows, and the keys of a tile that are its
    constexpr int kCopies = R::kCopies, kCols = R::kCols;
    const int row = quad * R::kWarpRows + (lane & (R::kWarpRows - 1));
    const int side = R::kHalf ? lane >> 4 : 0;     // of two threads that share a row
    const int copy = quad * R::kWarpRows / kRows;
    const int key0 = copy * R::kCopyKeys + side * kCols;
    const int qrow = row & (kRows - 1);            // query row
    const int warp_row = quad * R::kWarpRows & (kRows - 1);  // its warp's first
    uint32_t g = 0;      // tiles of this half so far
    uint32_t tile0 = 0;  // tiles of the pieces so far
    uint32_t pieces = 0;
    uint32_t passes = 0;  // of the join's buffer
    uint32_t sets = 0;    // groups of scales so far
    CfPiece u;
    while (next_piece(u)) {
      const int n_t = tiles_of(u, t);
      const int ctx = min(max(a.context_lens[u.r], 0), a.max_blocks * kBlockSize);
      const int pos0 = u.rt * kPos + row_tile * kCfPos;  // first query of the row tile
      const int live_rows = (min(pos0 + kCfPos, a.q_len) - pos0) * kGroup;
      const bool warp_live = warp_row < live_rows;
      const int first_key = ctx - a.q_len + pos0 + 1;    // keys that query 0 of the row tile sees
      const int seen = first_key + (qrow >> 2);          // that this row sees (<= 0: none)
      const int warp_seen = first_key + (warp_row >> 2);  // its warp's first row
      const uint32_t qb = q_slot(pieces, t);
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_full[qb], q_phase(pieces)));
      ++pieces;
      if (!ok) break;
      const float c = reinterpret_cast<const float*>(smem + S::kOffSigma)[qb * kCfRows + row];
      if constexpr (kWide) {
        // the queries' high parts to tensor memory: S is bound by what its
        // operands read of shared memory (with all of them there, 0.84 ms for 4 x
        // 2000 queries behind 4000 to 8000 tokens)
        const uint8_t* q = smem + S::kOffQ + qb * 2 * kCfPartBytes + row * 128;
        uint32_t w[32];
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const uint4 x = *reinterpret_cast<const uint4*>(q + ((ch ^ (row & 7)) << 4));
          w[4 * ch] = x.x;
          w[4 * ch + 1] = x.y;
          w[4 * ch + 2] = x.z;
          w[4 * ch + 3] = x.w;
        }
        tc::tmem_st16u(scol + kCfColQ, w);
        tc::tmem_st16u(scol + kCfColQ + 16, w + 16);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        mbar_arrive(&bars->qt_full[t]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_empty[qb]);
      float m = -INFINITY;  // what the weights are taken against (see kCfTop)
      float l = 0.f;        // sum of w / vs, in the weights' unit
      // Scales come in groups of 8 tiles, so that a tile need not wait for them.
      const uint32_t set0 = sets;
      sets += (u.take + kCfGroupTiles - 1) / kCfGroupTiles;
      uint32_t set = set0;  // the present one
      auto enter = [&]() -> bool {
        return __all_sync(0xffffffffu,
                          mbar_wait(&bars->sc_full[set % kCfScaleGroups], (set / kCfScaleGroups) & 1));
      };
      auto leave = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->sc_empty[set % kCfScaleGroups]);
        ++set;
      };
      ok = enter();
      if (!ok) break;
      for (int j = 0; j < n_t; ++j, ++g) {
        const int in_piece = kWide ? j : 2 * j + t;
        const int tok = (u.begin + in_piece) * kCfTokens;
        if (set0 + in_piece / kCfGroupTiles != set) {
          leave();
          ok = enter();
          if (!ok) break;
        }
        // (`ok` stays warp-uniform: the loads below are warp-collective)
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[t], g & 1));
        if (!ok) break;
        // the blocks' ks, log2 vs, 1 / vs (read twice: registers are dearer)
        const float* sc = reinterpret_cast<const float*>(smem + S::kOffScale) +
                          (set % kCfScaleGroups * kCfGroupTiles + in_piece % kCfGroupTiles) * kCfScaleFloats +
                          key0 / kBlockSize;
        tc::fence_after_sync();
        if (warp_live) {
          float s[kCols];
          if constexpr (R::kHalf) {
            tc::tmem_ld16x2_16<kCols>(scol + copy * R::kCopyKeys, s);
          } else {
#pragma unroll
            for (int e = 0; e < kCols; e += 32) tc::tmem_ld32(scol + key0 + e, s + e);
          }
          tc::tmem_wait_ld();
          tc::fence_before_sync();
          mbar_arrive(&bars->s_free[t]);
          const uint32_t pcol = scol + kCfColP;
          auto store = [&](uint32_t col, const uint32_t* w) {
            if constexpr (R::kHalf) {
              tc::tmem_st16x2_4<kCols / 4>(col, w);
            } else if constexpr (kCols == 64) {
              tc::tmem_st16u(col, w);
            } else {
              tc::tmem_st8(col, w);
            }
          };
          if (warp_seen - tok - copy * R::kCopyKeys < R::kCopyKeys) {  // some row of the warp sees its keys in part
            const int lim = seen - tok - key0;
#pragma unroll
            for (int e = 0; e < kCols; ++e)
              if (e >= lim) s[e] = -INFINITY;
          }
          float mx = -INFINITY;
#pragma unroll
          for (int b = 0; b < kCols / kBlockSize; ++b) {
            float x = fmaxf(s[16 * b], s[16 * b + 1]);
#pragma unroll
            for (int e = 2; e < 16; e += 2) x = fmaxf(fmaxf(x, s[16 * b + e]), s[16 * b + e + 1]);
            mx = fmaxf(mx, fmaf(x, fmaxf(sc[b] * c, kCfLeast), sc[kCfTileBlocks + b]));  // (the factor is > 0)
          }
          if constexpr (R::kHalf) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const bool grow = mx - m > kCfTop;  // also true the first time a row sees a key
          const float m_new = grow ? __fsub_ru(mx, cf_start(kWide)) : m;  // (upwards: far from zero no weight above)
          const float alpha = grow ? exp2_approx(m - m_new) : 1.f;  // 0 while m is -inf
          if (__any_sync(0xffffffffu, grow && j > 0 && m != -INFINITY)) {
            // O holds weights taken against the old maxima: rescale this warp's rows
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_done[t][(g - 1) & 1], ((g - 1) >> 1) & 1));
            if (!ok) break;
            tc::fence_after_sync();
            if constexpr (R::kHalf) {
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) {
                float o[32];
                tc::tmem_ld16x2_32<64>(scol + kCfColO + 32 * cc, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                tc::tmem_st16x2_32<64>(scol + kCfColO + 32 * cc, o);
              }
            } else {
#pragma unroll
              for (int cc = 0; cc < 8; ++cc) {
                float o[16];
                tc::tmem_ld16(scol + kCfColO + 16 * cc, o);
                tc::tmem_wait_ld();
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
                tc::tmem_st16u(scol + kCfColO + 16 * cc, w);
              }
            }
            tc::tmem_wait_st();
          }
          l *= alpha;
          m = m_new;
          // The weights' exponents, y - m: y rounded as for the maximum, then the
          // difference, which is exact near m.  (Fused, y is not rounded and m is:
          // where scores reach 2^25 the largest weight was off by factors of 2 and
          // more and left its parts' range.  Chunks took 2 % less time, drafts as much.)
          const float less = m == -INFINITY ? 0.f : -m;
          auto weights_of = [&](int i, float kc, float lv) -> float2 {
            float2 y = __ffma2_rn(make_float2(s[i], s[i + 1]), make_float2(kc, kc), make_float2(lv, lv));
            y = __fadd2_rn(y, make_float2(less, less));
            return make_float2(exp2_approx(y.x), exp2_approx(y.y));
          };
          auto weights_free = [&]() {  // their place is free once the product before is done
            if (j > 0) {
              ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_done[t][(g - 1) & 1], ((g - 1) >> 1) & 1));
              tc::fence_after_sync();
            }
            return ok;
          };
          if constexpr (kWide) {
            uint32_t w[8 * kCfTileBlocks];
#pragma unroll
            for (int b = 0; b < kCfTileBlocks; ++b) {
              const float kc = fmaxf(sc[b] * c, kCfLeast), lv = sc[kCfTileBlocks + b];
              float2 acc = make_float2(0.f, 0.f);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 p = weights_of(16 * b + 2 * e, kc, lv);
                acc = __fadd2_rn(acc, p);
                w[8 * b + e] = cf_half2(p.x, p.y);
              }
              l = fmaf(acc.x + acc.y, sc[2 * kCfTileBlocks + b], l);
            }
            if (!weights_free()) break;
            tc::tmem_st16u(pcol, w);
            tc::tmem_st16u(pcol + 16, w + 16);
          } else {
            uint32_t hi[kCols / 4], mid[kCols / 4], lo[kCols / 4];
#pragma unroll
            for (int b = 0; b < kCols / kBlockSize; ++b) {
              const float kc = fmaxf(sc[b] * c, kCfLeast), lv = sc[kCfTileBlocks + b];
              float2 acc = make_float2(0.f, 0.f);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 p = weights_of(16 * b + 4 * e, kc, lv), q = weights_of(16 * b + 4 * e + 2, kc, lv);
                acc = __fadd2_rn(acc, p);
                acc = __fadd2_rn(acc, q);
                cf_weights(p.x, p.y, q.x, q.y, hi[4 * b + e], mid[4 * b + e], lo[4 * b + e]);
              }
              l = fmaf(acc.x + acc.y, sc[2 * kCfTileBlocks + b], l);
            }
            if (!weights_free()) break;
            const uint32_t at = pcol + copy * (R::kCopyKeys / 4);
            store(at, hi);
            store(at + kCfPartCols, mid);
            store(at + 2 * kCfPartCols, lo);
            if constexpr (kCopies > 1) {  // the other copy's keys: weights of zero
              const uint32_t zeros[kCols / 4] = {};
              const uint32_t other = pcol + (copy ^ 1) * (R::kCopyKeys / 4);
#pragma unroll
              for (int part = 0; part < 3; ++part) store(other + part * kCfPartCols, zeros);
            }
            if (ctx - tok < kCfTokens && (ctx & (kBlockSize - 1)) != 0) {
              // slots past the context may hold any code: V's rows there are
              // zeroed (a weight of zero is not enough)
              const uint32_t vp = 2 * (tile0 + in_piece) + 1;
              ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[vp % kSlots], (vp / kSlots) & 1));
              if (!ok) break;
              const int z0 = ctx - tok, z1 = (z0 + kBlockSize - 1) & ~(kBlockSize - 1);
              uint8_t* vt = smem + S::kOffRing + (vp % kSlots) * kCfTileBytes;
              for (int i = z0 * 8 + lane; i < z1 * 8; i += 32) reinterpret_cast<uint4*>(vt)[i] = make_uint4(0, 0, 0, 0);
              tc::fence_proxy_async_smem();
            }
          }
          tc::tmem_wait_st();
          tc::fence_before_sync();
          mbar_arrive(&bars->p_full[t][g & 1]);
        } else {
          mbar_arrive(&bars->s_free[t]);
          mbar_arrive(&bars->p_full[t][g & 1]);
        }
      }
      tile0 += u.take;
      if (!ok) break;
      leave();
      if (set != sets) {  // (a last group of one tile, the other half's)
        ok = enter();
        if (!ok) break;
        leave();
      }
      if constexpr (R::kHalf) l += __shfl_xor_sync(0xffffffffu, l, 16);
      // ---- results ----
      if (n_t > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_done[t][(g - 1) & 1], ((g - 1) >> 1) & 1));
        if (!ok) break;
        tc::fence_after_sync();
      }
      const bool whole = u.take == u.n;
      const int64_t out_row0 = (static_cast<int64_t>(u.r) * a.q_len + pos0) * hq + u.kvh * kGroup;  // of query row 0
      const int64_t part_row0 =
          static_cast<int64_t>(2 * blockIdx.x + (u.begin == 0 ? 1 : 0)) * a.rows_slot + row_tile * kCfRows;
      if constexpr (kWide) {
        if (!warp_live) continue;
        const bool valid = qrow < live_rows;
        const float inv = l != 0.f ? 1.f / l : 0.f;  // (a NaN sum stays one)
        const int64_t out_row = out_row0 + static_cast<int64_t>(qrow >> 2) * hq + (qrow & 3);
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float o[32];
          tc::tmem_ld32(scol + kCfColO + 32 * cc, o);
          tc::tmem_wait_ld();
          if (valid && whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + out_row * kHeadDim + 32 * cc);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint4 w = make_uint4(0, 0, 0, 0);
              if (l != 0.f)
                w = make_uint4(pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv),
                               pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                               pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                               pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
              dst[e] = w;
            }
          } else if (valid) {
            float4* dst = reinterpret_cast<float4*>(a.part_o + (part_row0 + qrow) * kHeadDim + 32 * cc);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (valid && !whole) a.part_ml[part_row0 + qrow] = l != 0.f ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
      } else {
        // Join the two halves' copies: maxima and sums first, then 32 dims of
        // each thread a pass.  A thread joins 4 dims of up to kTake rows.
        constexpr int kParts = 2 * kCopies;          // partials of a row
        constexpr int kChunks = R::kHalf ? 16 : 8;   // of 4 dims, in a row of the buffer
        constexpr int kTake = kRows * kChunks / 256;
        float4* buf = reinterpret_cast<float4*>(smem + S::kOffExtra);
        const int who = t * R::kMma + row;
        auto written = [&]() -> bool {  // everyone's part of a pass is there
          mbar_arrive(&bars->join_full);
          return __all_sync(0xffffffffu, mbar_wait(&bars->join_full, passes & 1));
        };
        auto may_write = [&]() -> bool {  // everyone has read the pass before
          return passes == 0 || __all_sync(0xffffffffu, mbar_wait(&bars->join_free, (passes & 1) ^ 1));
        };
        auto read = [&]() {
          mbar_arrive(&bars->join_free);
          ++passes;
        };
        ok = may_write();
        if (!ok) break;
        reinterpret_cast<float2*>(buf)[who] = make_float2(m, l);
        ok = written();
        if (!ok) break;
        float f[kTake][kParts];
        const int ch = threadIdx.x & (kChunks - 1);
#pragma unroll
        for (int k = 0; k < kTake; ++k) {
          const int rr = (threadIdx.x + 256 * k) / kChunks;
          float2 ml[kParts];
          float mm = -INFINITY, sum = 0.f;
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            ml[q] = reinterpret_cast<const float2*>(buf)[q * kRows + rr];
            mm = fmaxf(mm, ml[q].x);
          }
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            f[k][q] = ml[q].y == 0.f ? 0.f : exp2_approx(ml[q].x - mm);  // (0: it saw nothing)
            sum = fmaf(ml[q].y, f[k][q], sum);
          }
          if (!whole && ch == 0 && rr < live_rows)
            a.part_ml[part_row0 + rr] = sum != 0.f ? make_float2(mm, sum) : make_float2(-INFINITY, 0.f);
          const float inv = whole ? (sum != 0.f ? 1.f / sum : 0.f) : 1.f;
#pragma unroll
          for (int q = 0; q < kParts; ++q) f[k][q] *= inv;
        }
        read();
#pragma unroll
        for (int cc = 0; cc < 32 / kChunks; ++cc) {
          ok = may_write();
          if (!ok) break;
          if (warp_live && n_t > 0) {
            float o[32];
            if constexpr (R::kHalf)
              tc::tmem_ld16x2_32<64>(scol + kCfColO + 32 * cc, o);
            else
              tc::tmem_ld32(scol + kCfColO + 32 * cc, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              buf[who * kChunks + side * 8 + (e ^ (row & 7))] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          ok = written();
          if (!ok) break;
          const int dim0 = 32 * cc + (ch >> 3) * 64;
#pragma unroll
          for (int k = 0; k < kTake; ++k) {
            const int rr = (threadIdx.x + 256 * k) / kChunks;
            if (rr >= live_rows) continue;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
              if (f[k][q] == 0.f) continue;  // nothing was written for it, or it adds nothing
              const float4 x = buf[(q * kRows + rr) * kChunks + (ch ^ (rr & 7))];
              o.x = fmaf(x.x, f[k][q], o.x);
              o.y = fmaf(x.y, f[k][q], o.y);
              o.z = fmaf(x.z, f[k][q], o.z);
              o.w = fmaf(x.w, f[k][q], o.w);
            }
            if (whole) {
              const int64_t out_row = out_row0 + static_cast<int64_t>(rr >> 2) * hq + (rr & 3);
              reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_row * kHeadDim + dim0)[ch & 7] =
                  make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
            } else {
              reinterpret_cast<float4*>(a.part_o + (part_row0 + rr) * kHeadDim + dim0)[ch & 7] = o;
            }
          }
          read();
        }
        if (!ok) break;
      }
      tc::fence_before_sync();  // O is read before the next piece's weights arrive
    }
    if (!ok && lane == 0) report(a.err, PKV_DEVERR_TIMEOUT);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of a job that was cut.  Block x of the grid looks at the
// cut where CTA x's share starts, and takes the job if that cut is its first;
// one warp per row, 4 dims a lane.
__global__ void __launch_bounds__(256) scaled_join_kernel(const ScaledArgs a, int32_t pos, int32_t job_cost) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x + 1;
  const CfCut cut = a.cuts[i];
  if (cut.into == 0) return;                      // no cut here
  const int start = cut.per * i - cut.into;       // where the job's cost begins
  if (start / cut.per != i - 1) return;           // cut earlier already
  const int pieces = (start + cut.n + job_cost - 1) / cut.per - (i - 1) + 1;
  // tiles of the job's k-th piece, in CTA i - 1 + k
  auto tile_at = [&](int cta) -> int { return min(max(cta * cut.per - start - job_cost, 0), cut.n); };
  if (tile_at(i) == 0 && pieces == 2) return;     // the cut fell before its first tile: one piece
  const int lane = threadIdx.x & 31;
  const int rows = min(pos, a.q_len - cut.rt * pos) * kGroup;
  const int hq = a.num_kv_heads * kGroup;
  for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < rows; row += gridDim.y * 8) {
    // a piece that begins the job lies in the second place of its CTA, others in the first
    const int first = tile_at(i) == 0 ? 1 : 0;
    auto at = [&](int k) -> int64_t {
      return static_cast<int64_t>(2 * (i - 1 + k) + (k == first ? 1 : 0)) * a.rows_slot + row;
    };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pieces - first == 2) {  // the usual cut
      float2 ml[2];
      float4 x[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ml[k] = a.part_ml[at(first + k)];
        x[k] = *reinterpret_cast<const float4*>(a.part_o + at(first + k) * kHeadDim + 4 * lane);
      }
      m = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (ml[k].y == 0.f) continue;  // it saw nothing, its O holds anything
        const float f = exp2_approx(ml[k].x - m);
        l = fmaf(ml[k].y, f, l);
        o.x = fmaf(x[k].x, f, o.x);
        o.y = fmaf(x[k].y, f, o.y);
        o.z = fmaf(x[k].z, f, o.z);
        o.w = fmaf(x[k].w, f, o.w);
      }
    } else {
      // 32 pieces at a time: lane k holds the k-th one's maximum and sum, and
      // what is summed so far is taken against the maximum so far
      constexpr int kFlight = 8;  // partials in flight
      for (int k0 = first; k0 < pieces; k0 += 32) {
        const int n = min(32, pieces - k0);
        float4 x[kFlight];
        auto fetch = [&](int b) {
#pragma unroll
          for (int k = 0; k < kFlight; ++k)
            if (b + k < n) x[k] = *reinterpret_cast<const float4*>(a.part_o + at(k0 + b + k) * kHeadDim + 4 * lane);
        };
        fetch(0);
        const float2 ml = lane < n ? a.part_ml[at(k0 + lane)] : make_float2(-INFINITY, 0.f);
        float top = ml.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float m_new = fmaxf(m, top);
        const float old = m == -INFINITY ? 0.f : exp2_approx(m - m_new);
        const float f = ml.y == 0.f ? 0.f : exp2_approx(ml.x - m_new);  // (0: it saw nothing, its O holds anything)
        float sum = ml.y * f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * old + sum;
        o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
        m = m_new;
        for (int b = 0; b < n; b += kFlight) {
          if (b > 0) fetch(b);
#pragma unroll
          for (int k = 0; k < kFlight; ++k) {
            const float g = __shfl_sync(0xffffffffu, f, (b + k) & 31);
            if (b + k >= n || g == 0.f) continue;
            o.x = fmaf(x[k].x, g, o.x);
            o.y = fmaf(x[k].y, g, o.y);
            o.z = fmaf(x[k].z, g, o.z);
            o.w = fmaf(x[k].w, g, o.w);
          }
        }
      }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t out_row = (static_cast<int64_t>(cut.r) * a.q_len + cut.rt * pos + (row >> 2)) * hq + cut.kvh * kGroup + (row & 3);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_row * kHeadDim)[lane] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

template <bool kWide, int kRows>
cudaError_t launch_cf(const ScaledArgs& a, int32_t grid, cudaStream_t stream) {
  static std::atomic<bool> done[64];  // per device; host threads may race on a first call
  auto kernel = paged_chunk_fp8_tc_kernel<kWide, kRows>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CfShape<kWide>::kSmem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  const int64_t rows = static_cast<int64_t>(a.num_blocks) * a.num_kv_heads * kBlockSize;
  CUtensorMap kmap, vmap;
  if (!make_pool_map_e4m3(&kmap, a.k_cache, rows) || !make_pool_map_e4m3(&vmap, a.v_cache, rows))
    return cudaErrorInvalidValue;
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kCfThreads), CfShape<kWide>::kSmem, stream,
                 1, kmap, vmap, a);
  if (e != cudaSuccess || grid == 1 || a.max_blocks <= kCfTileBlocks) return e;  // (a job of one tile is not cut)
  return launch_scaled_join(a, grid, kWide ? 2 * kCfPos : kCfPos, kCfJobCost, stream);
}

bool cf_wide(int32_t q_len) { return q_len > kCfPos; }

}  // namespace

cudaError_t launch_scaled_join(const ScaledArgs& a, int32_t grid, int32_t pos, int32_t job_cost, cudaStream_t stream) {
  // 8 rows a block at a time; a job of few rows is joined by one block
  const unsigned parts = (std::min(pos, a.q_len) * kGroup + 7) / 8;
  return launch_pdl(scaled_join_kernel, dim3(static_cast<unsigned>(grid - 1), parts), dim3(256), 0, stream, 1, a, pos,
                    job_cost);
}

int32_t chunk_scaled_grid(int32_t num_seqs, int32_t num_kv_heads, int32_t q_len, int32_t max_blocks, int32_t sm_count) {
  const int32_t pos = cf_wide(q_len) ? 2 * kCfPos : kCfPos;
  const int64_t jobs = static_cast<int64_t>(num_seqs) * num_kv_heads * ((q_len + pos - 1) / pos);
  const int64_t cost = jobs * ((max_blocks + kCfTileBlocks - 1) / kCfTileBlocks + kCfJobCost);  // at most
  // (shares are rounded up, so the last one may end behind the work)
  if (cost + int64_t{kCfMinShare} * sm_count > 0x7fffffff) return 0;
  return static_cast<int32_t>(std::min<int64_t>(sm_count, (cost + kCfMinShare - 1) / kCfMinShare));
}

int32_t chunk_scaled_rows(int32_t q_len) { return cf_wide(q_len) ? 2 * kCfRows : kGroup * q_len; }

cudaError_t launch_paged_chunk_fp8_tc(const ScaledArgs& a, int32_t grid, cudaStream_t stream) {
  if (cf_wide(a.q_len)) return launch_cf<true, 128>(a, grid, stream);
  const int32_t rows = kGroup * a.q_len;
  if (rows <= 32) return launch_cf<false, 32>(a, grid, stream);
  return rows <= 64 ? launch_cf<false, 64>(a, grid, stream) : launch_cf<false, 128>(a, grid, stream);
}

}  // namespace pkv
