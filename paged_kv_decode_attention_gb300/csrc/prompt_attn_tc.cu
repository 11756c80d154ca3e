// prompt_attn_tc.cu -- causal attention of whole prompts, packed one behind
// the other, on the 5th-generation tensor cores: the first step of a request
// ("Chapter 8: Inference Optimization", clxhxhhr.top/posts/4341, §8.1.1: the
// prefill computes K and V of all prompt tokens at once; §8.3.1 names the
// blockwise softmax used here).  K and V come straight from the projections,
// before they are stored in the cache.
//
// Mathematics: O_i = sum_{j <= i} w_ij V_j / sum_{j <= i} w_ij, w_ij =
// exp(scale q_i.k_j - m_i), evaluated over tiles of 64 keys with a running
// maximum and sum (FP32); S = Q K^T and O = P V with FP32 accumulators in
// tensor memory.
//
// Tiles are 64 keys: scores (64 columns), two buffers of weights (32 each) and
// O fill the 256 columns of a row tile.  The next scores are issued as soon as
// the softmax holds the present ones in registers, ahead of the product that
// waits for their weights, so neither side waits for the other's latency, and
// one commit tells the softmax that its next scores are there and that the
// weights' buffer is free.  What bounds it: the tensor pipe, 1280 cycles a
// tile and pair of row tiles (an MMA with N = 64 takes 48 cycles where its
// multiplications need 32, as it re-reads its 128-row operand), and for long
// prompts the power limit.  Measured, 32 query and 8 KV heads: 2 prompts of
// 16000 tokens 2.64 to 2.69 ms, 1.6 PFLOP/s, nine tenths of what a library's matrix
// product holds for seconds (with tiles of 128 keys and one buffer for scores and
// weights, one chain of S, softmax and P.V, 3.27; 64 keys, two such buffers, S
// two tiles ahead and after the product that frees its buffer 3.15).  64 prompts
// of 16 to 500 tokens 43.5 us (4.3 TB/s): 3.4 units a CTA, of which a start, a
// first tile and an end are not hidden, and a last round that most CTAs sit out.  (Results by four or eight warps of
// their own, as the softmax goes on: 54 us, as their registers are the
// softmax's.)
//
// A unit of work is (prompt, KV head, 256 rows): rows are query positions x
// the query heads of the KV head, so that a short prompt still fills them and
// the diagonal wastes little.  With G query heads to a KV head a row tile of
// 128 holds 128 / G positions (G that do not divide 128 leave a few rows
// unused).  The unit of a prompt's first positions costs one tile of keys,
// the next ones more: the i-th unit of every prompt costs about the same.  So
// the units are taken in falling order of i, by CTAs that stay (one per SM),
// forth and back over the grid, and no list has to be sorted.  A CTA passes
// over the prompts' bounds twice for each index at which their number changes:
// to count them, and on its way through them.  (4096 prompts of 16 to 200 tokens
// and one of 16000: 3.1 ms; with a count for every index and every search from
// the first prompt 14.6.)
//
// CTA = 12 warps:
//   warps 0-7: softmax, one thread per row (TMEM lane), one warpgroup for each
//             of the two row tiles.
//   warp 8  : TMA producer of K and V, into one ring of 16 KiB stages.
//   warps 9, 10: MMA issuers, one per row tile: while one tile's softmax runs,
//             the tensor cores work on the other's products.
//   warp 11 : finds the CTA's units, one ahead of the others, and loads Q.  (By
//             the producer of K and V, each row tile waits for the other's queries.)
#include <climits>
#include <cmath>
#include <cstddef>

#include "pkv_common.cuh"
#include "pkv_kernels.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kPaRows = 128;                           // rows of a row tile: TMEM lanes
constexpr int kPaTokens = 64;                          // keys of a tile
constexpr int kPaHalfBytes = kPaTokens * 128;          // 64 dims of a tile of K or V: 8 KiB
constexpr int kPaTileBytes = 2 * kPaHalfBytes;         // 16 KiB
constexpr int kPaQHalfBytes = kPaRows * 128;
constexpr int kPaQBytes = 2 * kPaQHalfBytes;           // a row tile of Q: 32 KiB
constexpr int kPaStages = 8;                           // ring of K and V tiles, in turn (10: no faster, 6: 20 % slower)
constexpr int kPaThreads = 384;
constexpr int kPaOffQ = 0;                             // 2 row tiles
constexpr int kPaOffRing = 2 * kPaQBytes;
constexpr int kPaOffOut = kPaOffRing + kPaStages * kPaTileBytes;  // results on their way out: 4 KiB a softmax warp
constexpr int kPaOutBytes = 32 * 128;
constexpr int kPaOffBar = kPaOffOut + 8 * kPaOutBytes;
constexpr int kPaSmem = kPaOffBar + 512;
constexpr uint32_t kPaTileCols = 256;                  // per row tile: S, two buffers of P, O
constexpr uint32_t kPaColP = 64;
constexpr uint32_t kPaPCols = kPaTokens / 2;           // 2 BF16 a column
constexpr uint32_t kPaColO = 128;
// Registers per thread: the launch's 168 x 384, moved from the issuing
// warpgroup to the two softmax warpgroups, which hold a tile's scores.
constexpr int kPaSoftmaxRegs = 208;
constexpr int kPaIssueRegs = 80;
static_assert((2 * kPaSoftmaxRegs + kPaIssueRegs) * 128 <= 168 * kPaThreads, "register split");
static_assert(kPaSmem <= 227 * 1024, "one CTA per SM");
// Log2 units: the maximum that the weights are taken against may lag by this
// much (BF16 weights and FP32 sums have the range), so O is rarely rescaled.
constexpr float kPaLag = 16.f;
constexpr float kPaLn2 = 0.6931471805599453f;

struct alignas(16) PaUnit {
  int32_t tok0;  // the prompt's first row
  int32_t len;   // its tokens; 0: no more units
  int32_t pos0;  // the unit's first position
  int32_t kvh;
};

struct PaBars {
  uint64_t full[kPaStages];
  uint64_t empty[kPaStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], s_free[2];  // per row tile: scores are there, are in registers
  uint64_t p_full[2][2];          // row tile, buffer
  uint64_t o_done[2][2];          // (two: nobody waits for each of them in turn)
  uint64_t u_full[2], u_empty[2];
  PaUnit unit[2];
  uint32_t tmem_base;
};
static_assert(sizeof(PaBars) <= 512 && offsetof(PaBars, unit) % 16 == 0, "barrier area");

template <int kRegs>
__device__ __forceinline__ void pa_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void pa_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// TMA tiled load of a 3-D box.
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// Key tiles that the positions up to `last` see.
__device__ __forceinline__ int pa_tiles(int last) { return last / kPaTokens + 1; }

__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attn_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map, const PromptArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  auto* bars = reinterpret_cast<PaBars*>(smem + kPaOffBar);
  // (through a broadcast, so that the compiler knows it to be uniform)
  auto uniform = [](int x) -> int { return __shfl_sync(0xffffffffu, x, 0); };
  const int warp = uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPaStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->s_free[t], 128);
      mbar_init(&bars->p_full[t][0], 128);
      mbar_init(&bars->p_full[t][1], 128);
      mbar_init(&bars->o_done[t][0], 1);
      mbar_init(&bars->o_done[t][1], 1);
      mbar_init(&bars->u_full[t], 1);
      mbar_init(&bars->u_empty[t], 11);  // every other warp
    }
    fence_barrier_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tc::prefetch_tensor_map(&q_map);
    tc::prefetch_tensor_map(&k_map);
    tc::prefetch_tensor_map(&v_map);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_wait();  // everything below may read what earlier grids in the stream write
  pdl_trigger();

  const uint32_t tmem = uniform(bars->tmem_base);
  const uint32_t sbase = uniform(smem_addr(smem));
  const int per_tile = a.pos_per_tile;
  const int per_unit = 2 * per_tile;
  bool ok = true;

  // The next unit of this warp's walk, or false at the end.
  uint32_t walked = 0;
  auto next_unit = [&](PaUnit& u) -> bool {
    const int slot = walked & 1;
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->u_full[slot], (walked >> 1) & 1));
    if (!ok) return false;
    const int4 w = *reinterpret_cast<const int4*>(&bars->unit[slot]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->u_empty[slot]);
    ++walked;
    u.tok0 = uniform(w.x);
    u.len = uniform(w.y);
    u.pos0 = uniform(w.z);
    u.kvh = uniform(w.w);
    return u.len > 0;
  };
  // key tiles of row tile t of a unit (0: it has no positions)
  auto tiles_of = [&](const PaUnit& u, int t) -> int {
    const int first = u.pos0 + t * per_tile;
    return first < u.len ? pa_tiles(min(first + per_tile, u.len) - 1) : 0;
  };

  if (warp >= 8) {
    pa_regs_down<kPaIssueRegs>();
    if (warp == 11) {
      // ---------------------------- the units ----------------------------
      auto bounds = [&](int s, int& b, int& n) {
        const int lo = a.cu_seqlens[s], hi = a.cu_seqlens[s + 1];
        b = min(max(lo, 0), a.num_tokens);
        n = max(min(max(hi, 0), a.num_tokens) - b, 0);
        return lo < 0 || hi > a.num_tokens || hi < lo;
      };
      auto units_of = [&](int s) -> int {
        if (s >= a.num_seqs) return 0;
        int b, n;
        bounds(s, b, n);
        return (n + per_unit - 1) / per_unit;
      };
      int first32 = 0, most = 0;  // of the first 32 prompts, one a lane; of the longest prompt
      for (int s0 = 0; s0 < a.num_seqs; s0 += 32) {
        const int n = units_of(s0 + lane);
        if (s0 == 0) first32 = n;
        most = max(most, n);
        if (blockIdx.x == 0 && s0 + lane < a.num_seqs) {
          int b, x;
          if (bounds(s0 + lane, b, x)) report(a.err, PKV_DEVERR_SEQLENS);
        }
      }
      most = __reduce_max_sync(0xffffffffu, most);
      // prompts with a unit of index i; `same`: the least index with as many
      int same = 0;
      auto count = [&](int i) -> int {
        int c = __popc(__ballot_sync(0xffffffffu, first32 > i));
        int below = first32 > i ? 0 : first32;
#pragma unroll 4
        for (int s0 = 32; s0 < a.num_seqs; s0 += 32) {
          const int n = units_of(s0 + lane);
          c += __popc(__ballot_sync(0xffffffffu, n > i));
          below = max(below, n > i ? 0 : n);
        }
        same = __reduce_max_sync(0xffffffffu, below);
        return c;
      };
      uint32_t loaded[2] = {0, 0};
      // a unit's queries, once the row tile's last product with those before is done
      const uint64_t once = l2_policy_evict_first();
      const uint32_t q_bytes = static_cast<uint32_t>(per_tile) * a.group * 256;
      auto queries = [&](const PaUnit& u, uint32_t k) {
        if (lane == 0) {
          for (int t = 0; t < 2 && ok; ++t) {
            if (k > 0) ok = mbar_wait(&bars->q_empty[t], (k & 1) ^ 1);
            if (!ok) break;
            uint8_t* dst = smem + kPaOffQ + t * kPaQBytes;
            const int tok = u.tok0 + u.pos0 + t * per_tile;  // (past the last token: zeros)
            mbar_arrive_expect_tx(&bars->q_full[t], q_bytes);
            tma_load_3d(dst, &q_map, 0, u.kvh * a.group, tok, &bars->q_full[t], once);
            tma_load_3d(dst + kPaQHalfBytes, &q_map, 64, u.kvh * a.group, tok, &bars->q_full[t], once);
            loaded[t] = k + 1;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      };
      int index = most - 1;  // of the units in turn
      int64_t before = 0;    // (prompt, index) pairs ahead of this index
      int here = index >= 0 ? count(index) : 0;
      int from = 0, passed = 0;  // the search resumes at prompt `from`, with so many of this index ahead of it
      PaUnit was{0, 0, 0, 0};
      for (uint32_t round = 0;; ++round) {
        const int64_t w = static_cast<int64_t>(round) * gridDim.x +
                          ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        const int64_t rank = w / a.num_kv_heads;
        while (index >= 0 && rank >= before + here) {
          before += here;
          --index;
          if (index < same) here = index >= 0 ? count(index) : 0;
          from = passed = 0;
        }
        PaUnit u{0, 0, 0, 0};
        if (index >= 0) {
          // the (rank - before)-th prompt that has a unit of this index
          const int nth = static_cast<int>(rank - before);
          for (; from < a.num_seqs; from += 32) {
            const uint32_t has = __ballot_sync(0xffffffffu, (from == 0 ? first32 : units_of(from + lane)) > index);
            const int c = __popc(has);
            if (nth < passed + c) {
              const int s = from + __fns(has, 0, nth - passed + 1);
              bounds(s, u.tok0, u.len);
              u.pos0 = index * per_unit;
              u.kvh = static_cast<int>(w - rank * a.num_kv_heads);
              break;
            }
            passed += c;
          }
        }
        const int slot = round & 1;
        if (round >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&bars->u_empty[slot], ((round >> 1) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          bars->unit[slot] = u;
          mbar_arrive(&bars->u_full[slot]);
        }
        __syncwarp();
        if (round > 0) queries(was, round - 1);
        if (!ok || u.len == 0) break;
        was = u;
      }
      if (!ok && lane == 0) {
        report(a.err, PKV_DEVERR_TIMEOUT);
        // copies under way must land before shared memory is released
        for (int t = 0; t < 2; ++t)
          if (loaded[t] > 0) mbar_wait(&bars->q_full[t], (loaded[t] - 1) & 1);
      }
      __syncwarp();
    } else if (warp == 8) {
      // ---------------------------- TMA producer ----------------------------
      const uint64_t keep = l2_policy_evict_last();
      uint32_t filled = 0;  // ring stages so far
      PaUnit u;
      auto ring = [&](const CUtensorMap* map, int tok, int kvh) {
        const int st = filled % kPaStages;
        if (filled >= kPaStages) ok = ok && mbar_wait(&bars->empty[st], ((filled / kPaStages) & 1) ^ 1);
        if (!ok) return;
        uint8_t* dst = smem + kPaOffRing + st * kPaTileBytes;
        mbar_arrive_expect_tx(&bars->full[st], kPaTileBytes);
        tma_load_3d(dst, map, 0, kvh, tok, &bars->full[st], keep);
        tma_load_3d(dst + kPaHalfBytes, map, 64, kvh, tok, &bars->full[st], keep);
        ++filled;
      };
      while (next_unit(u)) {
        const int n = max(tiles_of(u, 0), tiles_of(u, 1));
        if (lane == 0) {
          for (int j = 0; j < n && ok; ++j) {
            ring(&k_map, u.tok0 + j * kPaTokens, u.kvh);
            if (ok) ring(&v_map, u.tok0 + j * kPaTokens, u.kvh);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      if (lane == 0) {
        if (!ok) {
          report(a.err, PKV_DEVERR_TIMEOUT);
          // copies under way must land before shared memory is released
          for (uint32_t f = filled > kPaStages ? filled - kPaStages : 0; f < filled; ++f)
            mbar_wait(&bars->full[f % kPaStages], (f / kPaStages) & 1);
        }
      }
      __syncwarp();
    } else {
      // ---------------------------- MMA issuers ----------------------------
      constexpr uint32_t kIdS = tc::idesc_bf16_f32(kPaRows, kPaTokens, false, false);
      constexpr uint32_t kIdO = tc::idesc_bf16_f32(kPaRows, kHeadDim, false, true);
      const int t = warp - 9;
      const bool leader = lane == 0;
      const uint32_t scol = tmem + t * kPaTileCols;
      const uint64_t q_desc = tc::smem_desc(sbase + kPaOffQ + t * kPaQBytes, 16, 1024);
      const uint64_t k_desc = tc::smem_desc(sbase + kPaOffRing, 16, 1024);
      const uint64_t v_desc = tc::smem_desc(sbase + kPaOffRing, kPaHalfBytes, 1024);
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity));
      };
      // both barriers tried before either result is looked at
      auto wait2 = [&](uint64_t* x, uint32_t xp, uint64_t* y, uint32_t yp) -> bool {
        const bool rx = mbar_try_wait(x, xp), ry = mbar_try_wait(y, yp);
        return __all_sync(0xffffffffu, (rx || mbar_wait(x, xp)) && (ry || mbar_wait(y, yp)));
      };
      // S of the K tile in stage st
      auto issue_s = [&](uint32_t st, bool last) {
        const uint64_t kd = k_desc + st * (kPaTileBytes >> 4);
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma_bf16(scol, q_desc + (((kk >> 2) * kPaQHalfBytes + 32 * (kk & 3)) >> 4),
                         kd + (((kk >> 2) * kPaHalfBytes + 32 * (kk & 3)) >> 4), kIdS, kk > 0);
          tc::commit(&bars->s_full[t]);
          if (last) tc::commit(&bars->q_empty[t]);  // the next unit's queries may come
        }
        __syncwarp();
      };
      // O += P V, P in buffer buf, V in stage st
      auto issue_pv = [&](int buf, uint32_t st, bool first) {
        const uint32_t p = scol + kPaColP + buf * kPaPCols;
        const uint64_t vd = v_desc + st * (kPaTileBytes >> 4);
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_bf16_tmem_a(scol + kPaColO, p + 8 * kk, vd + kk * (2048 >> 4), kIdO, (!first || kk > 0) ? 1u : 0u);
          tc::commit(&bars->o_done[t][buf]);
        }
        __syncwarp();
      };
      // A place in the ring: K tiles at even places, V tiles at odd ones.
      struct Place {
        uint32_t st = 0, ph = 0;
        __device__ __forceinline__ void step(uint32_t n) {
          st += n;
          if (st >= kPaStages) {
            st -= kPaStages;
            ph ^= 1;
          }
        }
      };
      // Stages go back by plain arrivals once a later wait has shown that the
      // products that read them are done.
      auto give_back = [&](uint32_t st) {
        if (leader) mbar_arrive(&bars->empty[st]);
      };
      // the place `tiles` tiles before
      auto before = [](const Place& p, uint32_t tiles) -> uint32_t {
        return p.st >= 2 * tiles ? p.st - 2 * tiles : p.st + kPaStages - 2 * tiles;
      };
      Place k, v;  // of the present tile's K and V
      v.step(1);
      uint32_t g = 0;  // tiles of this row tile so far
      uint32_t units = 0;
      PaUnit u;
      while (next_unit(u)) {
        const int n_t = tiles_of(u, t);
        const int n = max(tiles_of(u, 0), tiles_of(u, 1));
        ok = wait(&bars->q_full[t], units & 1);
        ++units;
        if (n_t > 0 && ok) {
          ok = wait(&bars->full[k.st], k.ph);
          if (ok) issue_s(k.st, n_t == 1);
        }
        for (int j = 0; j < n_t && ok; ++j, ++g) {
          const uint32_t k_now = k.st;
          k.step(2);
          // The scores are in registers.  (They were committed after the
          // product of two tiles before, so that is done too.)
          ok = j + 1 < n_t ? wait2(&bars->full[k.st], k.ph, &bars->s_free[t], g & 1) : wait(&bars->s_free[t], g & 1);
          if (!ok) break;
          give_back(k_now);
          if (j >= 2) give_back(before(v, 2));
          if (j + 1 < n_t) issue_s(k.st, j + 2 == n_t);
          ok = wait2(&bars->full[v.st], v.ph, &bars->p_full[t][g & 1], (g >> 1) & 1);
          if (!ok) break;
          issue_pv(g & 1, v.st, j == 0);
          v.step(2);
        }
        // the last two tiles' V, once their products are done
        for (int back = min(n_t, 2); back > 0 && ok; --back) {
          ok = wait(&bars->o_done[t][(g - back) & 1], ((g - back) >> 1) & 1);
          if (ok) give_back(before(v, back));
        }
        if (n_t == 0 && ok && leader) mbar_arrive(&bars->q_empty[t]);
        for (int j = n_t; j < n && ok; ++j) {  // tiles that only the other row tile reads
          ok = wait(&bars->full[k.st], k.ph);
          if (ok) give_back(k.st);
          ok = ok && wait(&bars->full[v.st], v.ph);
          if (ok) give_back(v.st);
          k.step(2);
          v.step(2);
        }
        if (!ok) break;
      }
      if (!ok && leader) report(a.err, PKV_DEVERR_TIMEOUT);
      __syncwarp();
    }
  } else {
    // ---------------------------- softmax ----------------------------
    pa_regs_up<kPaSoftmaxRegs>();
    const int t = warp >> 2;
    const int quad = warp & 3;  // TMEM sub-partition of this warp
    const int row = quad * 32 + lane;
    const int tid = threadIdx.x & 127;
    const uint32_t scol = tmem + (static_cast<uint32_t>(quad * 32) << 16) + t * kPaTileCols;
    const int row_pos = row / a.group;        // position within the row tile
    const int row_head = row - row_pos * a.group;
    const int warp_pos = quad * 32 / a.group;  // the warp's first row's
    const float c = a.scale_log2;              // > 0: the max of raw scores scales to the max of scaled ones
    const int hq = a.num_kv_heads * a.group;
    uint8_t* stage = smem + kPaOffOut + warp * kPaOutBytes;
    uint32_t g = 0;       // tiles of this row tile so far
    uint32_t place = 1;   // ring place of the present tile's V
    PaUnit u;
    while (next_unit(u)) {
      const int n_t = tiles_of(u, t);
      const int n = max(tiles_of(u, 0), tiles_of(u, 1));
      const int pos = u.pos0 + t * per_tile + row_pos;
      const bool valid = row_pos < per_tile && pos < u.len;
      float m = -INFINITY;  // scaled max the weights are taken against (lags the true max by < 2^16)
      float l = 0.f;        // the sum of the weights
      for (int j = 0; j < n_t; ++j, ++g) {
        const int buf = g & 1;
        const int tok = j * kPaTokens;
        // (`ok` stays warp-uniform: the loads below are warp-collective)
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[t], g & 1));
        if (!ok) break;
        tc::fence_after_sync();
        float s[64];  // raw scores
        tc::tmem_ld32(scol, s);
        tc::tmem_ld32(scol + 32, s + 32);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        mbar_arrive(&bars->s_free[t]);
        if (u.pos0 + t * per_tile + warp_pos + 1 - tok < kPaTokens) {  // some row of the warp sees the tile in part
          const int lim = pos + 1 - tok;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= lim) s[e] = -INFINITY;
        }
        float mx;
        {
          float t8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) t8[e] = fmaxf(fmaxf(s[e], s[e + 8]), s[e + 16]);
#pragma unroll
          for (int e = 0; e < 8; ++e) t8[e] = fmaxf(fmaxf(t8[e], s[e + 24]), s[e + 32]);
#pragma unroll
          for (int e = 0; e < 8; ++e) t8[e] = fmaxf(fmaxf(t8[e], s[e + 40]), fmaxf(s[e + 48], s[e + 56]));
          mx = fmaxf(fmaxf(fmaxf(t8[0], t8[1]), fmaxf(t8[2], t8[3])), fmaxf(fmaxf(t8[4], t8[5]), fmaxf(t8[6], t8[7])));
        }
        mx *= c;
        const bool grow = mx > m + kPaLag;  // also true the first time a row sees a key
        const float m_new = grow ? mx : m;
        const float alpha = grow ? exp2_approx(m - m_new) : 1.f;  // 0 while m is -inf
        if (__builtin_expect(__any_sync(0xffffffffu, grow && j > 0 && m != -INFINITY), 0)) {
          // O holds weights taken against the old maxima: rescale this warp's rows
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_done[t][(g - 1) & 1], ((g - 1) >> 1) & 1));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            float o[32];
            tc::tmem_ld32(scol + kPaColO + 32 * cc, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tc::tmem_st32(scol + kPaColO + 32 * cc, o);
          }
          tc::tmem_wait_st();
        }
        l *= alpha;
        m = m_new;
        if (__builtin_expect(u.len - tok < kPaTokens, 0)) {
          // rows of V behind the prompt (weight 0, but they may hold anything): zero them
          const uint32_t vp = place + 2 * j;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[vp % kPaStages], (vp / kPaStages) & 1));
          if (!ok) break;
          uint8_t* vt = smem + kPaOffRing + (vp % kPaStages) * kPaTileBytes;
          for (int i = (u.len - tok) * 16 + tid; i < kPaTokens * 16; i += 128)
            *reinterpret_cast<uint4*>(vt + ((i & 8) ? kPaHalfBytes : 0) + (i >> 4) * 128 + (i & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async_smem();  // before the product that the weights' arrival lets go
        }
        // Exponents in one fused multiply-add: its product is not rounded and m is, so
        // the largest weight is 2^(half a step of m), which FP32 holds up to 2^31.
        // (Differences of raw scores times c, right for any: 1 to 2 % more time.)
        const float nm = (m == -INFINITY) ? 0.f : -m;
        const float2 c2 = make_float2(c, c);
        const float2 nm2 = make_float2(nm, nm);
        float2 acc2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // the weights, 2 BF16 per 32-bit column (their buffer's last product is done: see the issuers)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __ffma2_rn(make_float2(s[32 * cc + 2 * e], s[32 * cc + 2 * e + 1]), c2, nm2);
            const float p0 = exp2_approx(x.x);
            const float p1 = exp2_approx(x.y);
            acc2[e & 1] = __fadd2_rn(acc2[e & 1], make_float2(p0, p1));
            pk[e] = pack_bf16x2(p0, p1);
          }
          tc::tmem_st16u(scol + kPaColP + buf * kPaPCols + 16 * cc, pk);
        }
        l += (acc2[0].x + acc2[0].y) + (acc2[1].x + acc2[1].y);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        mbar_arrive(&bars->p_full[t][buf]);
      }
      place += 2 * n;
      if (!ok) break;
      if (n_t == 0) continue;
      // ---- results ----
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_done[t][(g - 1) & 1], ((g - 1) >> 1) & 1));
      if (!ok) break;
      tc::fence_after_sync();
      const float inv = 1.f / l;  // (a row sees its own key: l > 0, or NaN)
      // Results leave as whole 128-byte lines, 64 dims of the warp's rows at a
      // time: a thread's own row in pieces costs 32 separate lines an
      // instruction (3000 to 4000 cycles a unit; 64 short prompts 49 us).
      const int64_t row0 = static_cast<int64_t>(u.tok0 + u.pos0 + t * per_tile) * hq + u.kvh * a.group;
      const int mine = valid ? row_pos * hq + row_head : -1;  // row of the output, from row0
      uint8_t* out0 = static_cast<uint8_t*>(a.out) + row0 * (kHeadDim * 2) + (lane & 7) * 16;
      int to[8];  // the rows that this lane stores a piece of
#pragma unroll
      for (int i = 0; i < 8; ++i) to[i] = __shfl_sync(0xffffffffu, mine, 4 * i + (lane >> 3));
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        float o[64];
        tc::tmem_ld32(scol + kPaColO + 64 * pass, o);
        tc::tmem_ld32(scol + kPaColO + 64 * pass + 32, o + 32);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)  // 16-byte chunk e of row r sits at chunk e ^ (r % 8)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv), pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                         pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                         pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
        __syncwarp();
        uint4 w[8];  // (all read before the first is stored: the compiler cannot know that they do not overlap)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3);
          w[i] = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (to[i] >= 0) *reinterpret_cast<uint4*>(out0 + static_cast<int64_t>(to[i]) * (kHeadDim * 2) + 128 * pass) = w[i];
        }
        __syncwarp();
      }
      if (valid && a.lse != nullptr) a.lse[row0 + mine] = (m + log2f(l)) * kPaLn2;
      tc::fence_before_sync();  // O is read before the next unit's weights arrive
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

cudaError_t allow_smem_pa() {
  static std::atomic<bool> done[64];  // per device; host threads may race on a first call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(prompt_attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPaSmem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& args, int32_t sm_count, cudaStream_t stream) {
  PromptArgs a = args;
  a.pos_per_tile = kPaRows / a.group;
  CUtensorMap qmap, kmap, vmap;
  const int32_t hq = a.num_kv_heads * a.group;
  if (!make_packed_map(&qmap, a.q, a.num_tokens, hq, a.q_stride, a.group, a.pos_per_tile) ||
      !make_packed_map(&kmap, a.k, a.num_tokens, a.num_kv_heads, a.k_stride, 1, kPaTokens) ||
      !make_packed_map(&vmap, a.v, a.num_tokens, a.num_kv_heads, a.v_stride, 1, kPaTokens))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem_pa();
  if (e != cudaSuccess) return e;
  // units: a prompt of n tokens has ceil(n / per_unit), so at most this many
  const int64_t per_unit = 2 * a.pos_per_tile;
  const int64_t most = (a.num_tokens / per_unit + a.num_seqs) * a.num_kv_heads;
  const int64_t grid = most < sm_count ? most : sm_count;
  return launch_pdl(prompt_attn_tc_kernel, dim3(static_cast<unsigned>(grid)), dim3(kPaThreads), kPaSmem, stream, 1,
                    qmap, kmap, vmap, a);
}

}  // namespace pkv
