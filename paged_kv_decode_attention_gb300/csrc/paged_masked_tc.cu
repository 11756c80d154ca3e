// paged_masked_tc.cu -- attention of several query positions per request
// under a mask other than the plain causal one, on the 5th-generation tensor
// cores, over a paged BF16 KV cache:
//
//   tree   : the last n tokens of the context are drafted tokens; draft i sees
//            every committed token and the drafts whose bits are set in its
//            mask row (its ancestors and itself).  "Chapter 8: Inference
//            Optimization" (clxhxhhr.top/posts/4341), §8.5.2: verifying several
//            drafted positions reads the same KV as one decode step.
//   window : the query at position p sees the keys p - W + 1 .. p and the first
//            `num_sinks` tokens; blocks that no query of the call sees are
//            neither read nor looked up.
//
// Mathematics: softmax over the visible keys, evaluated tile by tile with a
// running maximum and sum (FP32), S = Q K^T and O = P V with FP32 accumulators
// in tensor memory.  A mask is a 64-bit word per (row, 64 keys), computed once
// per tile and only for the tiles that some row of the CTA sees partly.
//
// Rows of a CTA = query positions x the 4 query heads of one KV head, so each
// K/V byte is read once for all of them.  What bounds it: HBM up to about 32
// positions; beyond, shared memory and the tensor pipe together: an MMA with
// N = 64 re-reads its 128-row A operand for every 64 keys and takes 48 cycles
// where its multiplications need 32, so S of a 64-token tile costs 384 cycles
// per row tile and P.V (A in tensor memory, N = 128) 256.  K/V tiles are 64
// tokens in both shapes: two buffers of scores, then O, fill the 256 columns
// of a row tile, and the second buffer (S two tiles ahead of the P.V that is
// under way) is worth more than S with N = 128 from a single buffer (replayed,
// in the version that compared them, 16 trees of 61 positions: 102 us against
// 114; 2000-token chunks: 390 against 480).  Half of the queries in tensor
// memory, with one buffer each for S and P, took 110 and 421 us there: an MMA
// whose A lies there is not faster at N = 64.
//   kQTiles 1: 128 rows (32 positions), 2 CTAs per SM.  The wait of one CTA
//              (first tiles, softmax latency, epilogue) is filled by the
//              other.  P.V carries the weights as a BF16 part plus the BF16
//              rounding of the remainder (about 2^-17 relative): the tensor
//              cores have the time, HBM is the bound.
//   kQTiles 2: 256 rows (64 positions), 1 CTA per SM; each row tile has its
//              own MMA warp, and while one's softmax runs the tensor cores
//              work on the other's products.  The weights enter P.V rounded
//              to BF16, 2^-8 relative at most.  Over many keys of like weight
//              the errors average out (0.0023 of the output's norm against
//              0.0017 from the output's own rounding).  Where one key holds
//              most of the weight they do not: with a maximum that lags (by
//              up to 2^16) its weight need not be 1, and the sum is that of
//              the unrounded weights, so up to 2^-8 reaches the output.  In
//              the version above, the remainder's products took 150 and 548 us
//              for 102 and 390, sums of the rounded weights 111 and 421.
//
// CTA = 4 + 4 kQTiles warps:
//   warps 0, 2: TMA producers of K and of V (16 x 64 boxes, 128-byte
//             swizzle, one per block and 64-dim half; blocks past the range
//             arrive as zeros).
//   warps 1, 3: MMA issuers, one per row tile (warp 3 idles in kQTiles 1).
//   warps 4..: softmax, one thread per row (TMEM lane).  Warps whose rows are
//             all padding only keep the barriers in step.
//
// Splits of a long context come together in one of three ways (MaskedMode);
// up to 8 of them form a cluster and merge through distributed shared memory
// (one request of 26 positions over 600 tokens: 8.4 us in one launch).
//
// Measured (32 query and 8 KV heads, BF16, one GB300; replayed from a graph
// over three sets of inputs / through the public call, one after another):
//   tree, 37 requests x 16 positions after about 2,100 tokens
//              53 / 54 to 55 us: 6.4 TB/s
//   tree, 16 x 61 positions after about 8,300 tokens
//              99 to 102 / 110 to 117 us: 5.6 TB/s, tensor pipe 73.5 % of the
//              active cycles (88 % on the busiest SM)
//   window 2000 + 4 sinks, 64 single queries
//              43 / 44 us: 5.2 TB/s; the tail of unequal lengths is what is left
//   window 4096 + 4 sinks, 4 chunks of 2000
//              355 to 377 / 383 to 390 us: 1380 cycles a tile and pair of row
//              tiles where the pipe needs 1280, and some 5 % around a unit
//              (kRounds; one unit per CTA 395, replayed)
#include <algorithm>
#include <climits>
#include <cmath>

#include "pkv_common.cuh"
#include "pkv_kernels.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

// Log2 units: weights stay below 2^16.  FP32 sums and BF16 weights have the
// range; a tile of few keys first (sinks) would make a bound of 2^8 rescale
// now and then (470 cycles each).
constexpr float kRescaleThreshold = 16.f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRowsPerTile = 128;                          // TMEM lanes
constexpr int kPosPerTile = kRowsPerTile / kGroup;         // query positions of a row tile: 32
constexpr int kQTileBytes = kRowsPerTile * kHeadDim * 2;   // 32 KiB, two 64-dim halves
constexpr int kQHalfBytes = kQTileBytes / 2;

// kTwoQ: two query buffers, so that the next unit's queries come while the
// present one is worked on (three stages a ring are as good as five for that).
template <int kQTiles, bool kTwoQ = false>
struct Shape {
  static constexpr int kQBufs = kTwoQ ? 2 : 1;
  static constexpr int kTileBlocks = kMaskedTileBlocks;
  static constexpr int kTileTokens = kTileBlocks * kBlockSize;  // 64
  static constexpr int kKStages = kQTiles == 1 || kTwoQ ? 3 : 5;
  static constexpr int kVStages = kQTiles == 1 ? 2 : (kTwoQ ? 3 : 5);
  static constexpr int kHalfBytes = kTileTokens * 128;
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kWarps = 4 + 4 * kQTiles;
  static constexpr int kThreads = kWarps * 32;
  // Registers per thread: the launch's share (65536 / (threads x CTAs)) is
  // moved from the four issuing warps to the softmax warps, which hold a
  // tile's scores; the sum stays within what the block was launched with.
  static constexpr int kLaunchRegs = kQTiles == 1 ? 128 : 168;
  static constexpr int kIssueRegs = kQTiles == 1 ? 64 : 80;
  static constexpr int kSoftmaxRegs = kQTiles == 1 ? 192 : 208;
  static_assert((kIssueRegs + kQTiles * kSoftmaxRegs) * 128 <= kLaunchRegs * kThreads, "register split");
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kQBufs * kQTiles * kQTileBytes;
  static constexpr int kOffV = kOffK + kKStages * kStageBytes;
  static constexpr int kOffBar = kOffV + kVStages * kStageBytes;
  static constexpr int kSmem = kOffBar + 512;
  // kCluster: partial O [row][128] FP32 over the K and V rings once they are
  // drained, then (max, sum) per row
  static constexpr int kOffPartO = kOffK;
  static constexpr int kOffPartML = kOffPartO + kQTiles * kRowsPerTile * kHeadDim * 4;
  static_assert(kTwoQ || kOffPartML + kQTiles * kRowsPerTile * 8 <= kOffBar, "the partials fit in the rings");
  static constexpr uint32_t kColO = 2 * kTileTokens;          // two S/P buffers, then O (128 columns)
  static constexpr uint32_t kTileCols = kColO + kHeadDim;     // 256 columns per row tile
  static constexpr uint32_t kTmemCols = kQTiles * kTileCols;  // 256 or 512
  static constexpr bool kRemainder = kQTiles == 1;
  static constexpr int kCtasPerSm = kQTiles == 1 ? 2 : 1;
  static_assert(kSmem <= (kQTiles == 1 ? 113 : 227) * 1024, "shared memory per CTA");
};

template <int kQTiles, bool kTwoQ = false>
struct Bars {
  using S = Shape<kQTiles, kTwoQ>;
  uint64_t k_full[S::kKStages];
  uint64_t k_empty[S::kKStages];
  uint64_t v_full[S::kVStages];
  uint64_t v_empty[S::kVStages];
  uint64_t s_full[kQTiles][2];
  uint64_t p_full[kQTiles][2];
  uint64_t o_done[kQTiles][2];
  uint64_t q_full[kQTiles][S::kQBufs];  // per unit whose row tile has queries
  uint32_t tmem_base;
  int32_t request;              // longest_first: the request of this CTA
};
static_assert(sizeof(Bars<2>) <= 512 && sizeof(Bars<2, true>) <= 512, "barrier area");

// How the splits of one (row tile, KV head) come together.
enum class MaskedMode {
  kDirect,     // one split: BF16 out
  kRounds,     // the same, several units per CTA
  kWorkspace,  // FP32 partials to the workspace, merged by the combine kernel
  kCluster     // one thread-block cluster: merged through distributed shared memory
};

template <int kQTiles, MaskedMode kMode>
using ShapeOf = Shape<kQTiles, kMode == MaskedMode::kRounds && kQTiles == 2>;

// Move registers between warpgroups (all warps of one execute it).
template <int kRegs>
__device__ __forceinline__ void set_max_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void set_max_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// The x lowest bits (x may lie outside 0..64).
__device__ __forceinline__ uint64_t low_bits(int x) {
  return x <= 0 ? 0ull : (x >= 64 ? ~0ull : (1ull << x) - 1ull);
}

template <int kQTiles, MaskKind kMask, MaskedMode kMode>
__device__ __forceinline__ void paged_masked_tc_body(const CUtensorMap& k_map, const CUtensorMap& v_map,
                                                     const MaskedArgs& a) {
  constexpr bool kMany = kMode == MaskedMode::kRounds;
  using S = ShapeOf<kQTiles, kMode>;
  constexpr bool kTwoQ = S::kQBufs == 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  auto* bars = reinterpret_cast<Bars<kQTiles, kTwoQ>*>(smem + S::kOffBar);
  // Warp indexes, tile counts and addresses go through a broadcast so that the
  // compiler knows them to be uniform: the issuing warps' descriptors then
  // live in uniform registers, where the MMA instructions read them.
  auto uniform = [](int x) -> int { return __shfl_sync(0xffffffffu, x, 0); };
  const int warp = uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;

  // ---------------- set-up: barriers, TMEM (reads no input) ----------------
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kKStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], kQTiles);
    }
    for (int s = 0; s < S::kVStages; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], kQTiles);
    }
    for (int t = 0; t < kQTiles; ++t)
      for (int s = 0; s < 2; ++s) {
        mbar_init(&bars->s_full[t][s], 1);
        mbar_init(&bars->p_full[t][s], 128);
        mbar_init(&bars->o_done[t][s], 1);
      }
    for (int t = 0; t < kQTiles; ++t)
      for (int b = 0; b < S::kQBufs; ++b) mbar_init(&bars->q_full[t][b], 128);
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&bars->tmem_base, S::kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tensor_map(&k_map);
    tc::prefetch_tensor_map(&v_map);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_wait();  // everything below may read what earlier grids in the stream write
  pdl_trigger();

  // ---------------- the units of this CTA ----------------
  // A unit: up to kPos query positions of one request for one KV head (row
  // tile fastest, then KV head, then request), one per CTA.  kRounds: the grid
  // is what is resident at once and a CTA takes a unit per round, forth and
  // back over the grid; the rings run on, so that a unit's copies are under
  // way while the one before ends.
  constexpr int kPos = kPosPerTile * kQTiles;  // query positions per CTA
  constexpr bool kToOut = kMode == MaskedMode::kDirect || kMany;
  const int n_rt = (a.d.q_len + kPos - 1) / kPos;
  const uint32_t n_units = static_cast<uint32_t>(a.d.num_seqs) * a.d.num_kv_heads * n_rt;
  const int rounds = kMany ? (n_units + gridDim.x - 1) / gridDim.x : 1;
  const int split = blockIdx.y;
  const int hq = a.d.num_kv_heads * kGroup;
  const int cap = a.d.max_blocks * kBlockSize;
  const int t_first = split * a.tiles_per_split;  // first tile of this split
  struct Unit {
    int r, kvh, pos0;  // request, KV head, first query index
    int ctx;
    int n_new;    // queries of this request
    int base;     // position of query 0
    int n_pos;    // queries of this unit (<= 0: none)
    // keys [0, sink_blocks*16) and [first_block*16, key_end) are read; the rest is not looked up
    int sink_blocks, first_block, key_end, end_block, sink_tiles;
    int n_tiles;  // of this split
    int q_tiles;  // row tiles with queries (kQTiles 1: always 1)
  };
  // unit of a round, or false past the last one
  auto place = [&](int round, Unit& w) -> bool {
    uint32_t u = blockIdx.x;
    if constexpr (kMany) {
      u = static_cast<uint32_t>(round) * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      if (u >= n_units) return false;
    }
    int x = u / n_rt;
    w.pos0 = static_cast<int>(u - x * n_rt) * kPos;
    w.kvh = x % a.d.num_kv_heads;
    w.r = uniform(x / a.d.num_kv_heads);
    return true;
  };
  // what the unit reads
  auto tree_len = [&](int r) -> int {
    return kMask == MaskKind::kTree && a.tree_lens != nullptr ? a.tree_lens[r] : a.d.q_len;
  };
  auto measure = [&](Unit& w, int ctx, int n_new) {
    w.ctx = ctx;
    w.n_new = min(max(n_new, 0), a.d.q_len);
    if (w.ctx > cap && threadIdx.x == 0 && split == 0 && w.kvh == 0 && w.pos0 == 0) report(a.d.err, PKV_DEVERR_CONTEXT);
    w.ctx = min(max(w.ctx, 0), cap);
    w.base = w.ctx - w.n_new;
    w.n_pos = min(kPos, w.n_new - w.pos0);
    w.sink_blocks = w.first_block = w.key_end = 0;
    if (w.n_pos > 0 && w.ctx > 0) {
      if constexpr (kMask == MaskKind::kTree) {
        w.key_end = w.ctx;
      } else {
        const int p_first = w.base + w.pos0;
        w.key_end = max(p_first + w.n_pos, 0);  // the last query sees its own position
        const int first_key = max(0, max(p_first, 0) - a.window + 1);
        w.first_block = first_key / kBlockSize;
        w.sink_blocks = (min(a.num_sinks, first_key) + kBlockSize - 1) / kBlockSize;
        if (w.sink_blocks >= w.first_block) w.sink_blocks = w.first_block = 0;  // one contiguous range
      }
    }
    w.end_block = (w.key_end + kBlockSize - 1) / kBlockSize;
    w.sink_tiles = (w.sink_blocks + S::kTileBlocks - 1) / S::kTileBlocks;
    const int all_tiles =
        w.sink_tiles + (max(0, w.end_block - w.first_block) + S::kTileBlocks - 1) / S::kTileBlocks;
    w.n_tiles = uniform(min(all_tiles - t_first, a.tiles_per_split));
    w.q_tiles = uniform(w.n_pos > kPosPerTile ? 2 : 1);
  };

  // the first unit, before the roles part: every warp waits for its length once
  // (kRounds: each role measures its units when it comes to them; carrying the
  // first one over costs registers, 417 us instead of 366 for 4 chunks of 2000)
  Unit unit0{};
  if (!kMany) place(0, unit0);
  if (kMode == MaskedMode::kDirect && a.longest_first) {
    // More CTAs than fit at once: the requests with the most to read start
    // first, so that none of them is left for the end.  Place r = the number
    // of requests that come before it.
    int32_t* len = reinterpret_cast<int32_t*>(smem + S::kOffQ);  // [num_seqs, + up to 3], before the queries come here
    const int padded = (a.d.num_seqs + 3) & ~3;
    for (int i = threadIdx.x; i < padded; i += S::kThreads)
      len[i] = i < a.d.num_seqs ? min(a.d.context_lens[i], a.span) : INT_MIN;
    __syncthreads();
    for (int i = threadIdx.x; i < a.d.num_seqs; i += S::kThreads) {
      const int mine = len[i];
      int before = 0;
      for (int k = 0; k < padded; k += 4) {
        const int4 v = *reinterpret_cast<const int4*>(len + k);
        before += (v.x > mine || (v.x == mine && k < i)) + (v.y > mine || (v.y == mine && k + 1 < i)) +
                  (v.z > mine || (v.z == mine && k + 2 < i)) + (v.w > mine || (v.w == mine && k + 3 < i));
      }
      if (before == unit0.r) bars->request = i;
    }
    __syncthreads();
    unit0.r = uniform(bars->request);
  }
  // Its first block ids are read before the context length is known (ids past
  // the range are dropped later): one trip less before the copies.
  int ids0 = 0;
  if (!kMany && kMask == MaskKind::kTree && (warp == 0 || warp == 2))
    ids0 = a.d.block_tables[static_cast<int64_t>(unit0.r) * a.d.max_blocks +
                            min(t_first * S::kTileBlocks + lane, a.d.max_blocks - 1)];
  if (!kMany) measure(unit0, a.d.context_lens[unit0.r], tree_len(unit0.r));
  const bool softmax_warp = warp >= 4;
  const uint32_t tmem = uniform(bars->tmem_base);
  const uint32_t sbase = uniform(smem_addr(smem));
  bool ok = true;
  float2* part_ml = reinterpret_cast<float2*>(smem + S::kOffPartML);

  if (!softmax_warp) {
    set_max_regs_down<S::kIssueRegs>();
    if (warp == 0 || warp == 2) {
      // ---------------------------- TMA producers ----------------------------
      const bool is_v = warp == 2;
      const int stages = is_v ? S::kVStages : S::kKStages;
      uint64_t* full = is_v ? bars->v_full : bars->k_full;
      uint64_t* empty = is_v ? bars->v_empty : bars->k_empty;
      uint8_t* ring = smem + (is_v ? S::kOffV : S::kOffK);
      const CUtensorMap* map = is_v ? &v_map : &k_map;
      // read once, unless several row tiles of the request read the same blocks
      const uint64_t policy = n_rt > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
      const int oob_row = a.d.num_blocks * a.d.num_kv_heads * kBlockSize;  // first row past the pool
      int filled = 0;  // tiles so far
      for (int round = 0; round < rounds && ok; ++round) {
        Unit w = unit0;
        int first_ids = ids0;
        if (kMany) {
          if (!place(round, w)) continue;
          if (kMask == MaskKind::kTree)
            first_ids = a.d.block_tables[static_cast<int64_t>(w.r) * a.d.max_blocks + min(lane, a.d.max_blocks - 1)];
          measure(w, a.d.context_lens[w.r], tree_len(w.r));
        }
        const int32_t* table = a.d.block_tables + static_cast<int64_t>(w.r) * a.d.max_blocks;
        // logical block of entry i of the list of blocks (whole tiles of sinks,
        // then the window), or -1 for a hole or past the range.  Kept apart
        // from the table's entries, which may hold any value.
        auto logical = [&](int i) -> int {
          if (i >= w.n_tiles * S::kTileBlocks) return -1;
          i += t_first * S::kTileBlocks;
          const int sink_entries = w.sink_tiles * S::kTileBlocks;
          const int lb = i < sink_entries ? (i < w.sink_blocks ? i : INT_MAX) : w.first_block + i - sink_entries;
          return lb < w.end_block ? lb : -1;
        };
        // its pool row, given its block id
        auto row_of = [&](int lb, int blk) -> int {
          if (lb < 0) return oob_row;
          if (blk < 0 || blk >= a.d.num_blocks) {
            report(a.d.err, PKV_DEVERR_BLOCK_ID);
            blk = 0;
          }
          return (blk * a.d.num_kv_heads + w.kvh) * kBlockSize;
        };
        constexpr int kTilesPerChunk = 32 / S::kTileBlocks;
        int next_lb = logical(lane), nxt = first_ids;  // (a tree's were read above)
        if (kMask != MaskKind::kTree && next_lb >= 0) nxt = table[next_lb];
        int cur = row_of(next_lb, nxt);
        for (int j = 0; j < w.n_tiles && ok; ++j, ++filled) {
          const int in_chunk = j % kTilesPerChunk;
          if (in_chunk == 0) {  // the next chunk's ids, checked when they are used
            next_lb = logical((j + kTilesPerChunk) * S::kTileBlocks + lane);
            if (next_lb >= 0) nxt = table[next_lb];
          }
          const int yy = __shfl_sync(0xffffffffu, cur, in_chunk * S::kTileBlocks + ((lane >> 1) & (S::kTileBlocks - 1)));
          if (in_chunk == kTilesPerChunk - 1) cur = row_of(next_lb, nxt);
          const int st = filled % stages;
          if (filled >= stages) ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ((filled / stages) & 1) ^ 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[st], S::kStageBytes);
          __syncwarp();
          if (lane < 2 * S::kTileBlocks) {
            const int b = lane >> 1, c = lane & 1;
            tc::tma_load_2d(ring + st * S::kStageBytes + c * S::kHalfBytes + b * 2048, map, c * 64, yy, &full[st], policy);
          }
        }
      }
      if (lane == 0) {
        if (!ok) report(a.d.err, PKV_DEVERR_TIMEOUT);
        // the last tiles' copies must land before shared memory is released
        for (int j = max(0, filled - stages); j < filled; ++j) mbar_wait(&full[j % stages], (j / stages) & 1);
      }
    } else if (kQTiles == 2 || warp == 1) {
      // ---------------------------- MMA issuer ----------------------------
      // One warp per row tile, so that neither tile's products wait for the
      // other's weights.  The whole warp walks the loop and lane 0 issues.
      // Per tile: P.V as soon as its weights are there, then S two tiles ahead
      // (into the buffer that this P.V reads, so after its completion): the
      // softmax always has a scored tile to go on with.
      constexpr uint32_t kIdS = tc::idesc_bf16_f32(kRowsPerTile, S::kTileTokens, false, false);
      constexpr uint32_t kIdO = tc::idesc_bf16_f32(kRowsPerTile, kHeadDim, false, true);
      const uint64_t q_desc = tc::smem_desc(sbase + S::kOffQ, 16, 1024);
      const uint64_t k_desc = tc::smem_desc(sbase + S::kOffK, 16, 1024);
      const uint64_t v_desc = tc::smem_desc(sbase + S::kOffV, S::kHalfBytes, 1024);
      const bool leader = lane == 0;
      const int t = warp >> 1;  // warp 1 or 3
      const uint32_t tcol = tmem + t * S::kTileCols;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity));
      };
      // both barriers tried before either result is looked at
      auto wait2 = [&](uint64_t* x, uint32_t xp, uint64_t* y, uint32_t yp) -> bool {
        const bool rx = mbar_try_wait(x, xp), ry = mbar_try_wait(y, yp);
        return __all_sync(0xffffffffu, (rx || mbar_wait(x, xp)) && (ry || mbar_wait(y, yp)));
      };
      // Stages go back by plain arrivals once a later wait has shown that the
      // products that read them are done (a commit costs this warp 46 cycles).
      auto give_back = [&](uint64_t* bar) {
        if (leader) mbar_arrive(bar);
      };
      // S of the tile in K stage st, into buffer buf
      auto issue_s = [&](int buf, int st, int qb) {
        const uint32_t d = tcol + buf * S::kTileTokens;
        const uint64_t qd = q_desc + (qb * kQTiles + t) * (kQTileBytes >> 4);
        const uint64_t kd = k_desc + st * (S::kStageBytes >> 4);
        tc::fence_after_sync();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma_bf16(d, qd + (((kk >> 2) * kQHalfBytes + 32 * (kk & 3)) >> 4),
                         kd + (((kk >> 2) * S::kHalfBytes + 32 * (kk & 3)) >> 4), kIdS, kk > 0);
          tc::commit(&bars->s_full[t][buf]);
        }
        __syncwarp();
      };
      // O += P V, P in buffer buf (its BF16 parts, then their remainders), V in stage st
      auto issue_pv = [&](int buf, int st, bool first) {
        const uint32_t ptm = tcol + buf * S::kTileTokens;
        const uint64_t vd = v_desc + st * (S::kStageBytes >> 4);
        tc::fence_after_sync();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < (S::kRemainder ? 8 : 4); ++kk)
            tc::mma_bf16_tmem_a(tcol + S::kColO, ptm + 8 * kk, vd + (kk & 3) * (2048 >> 4), kIdO,
                                (!first || kk > 0) ? 1u : 0u);
          tc::commit(&bars->o_done[t][buf]);
        }
        __syncwarp();
      };
      uint32_t g = 0;               // tiles of this row tile so far
      int units = 0;                // of this row tile so far
      int ahead_ctx = 0, ahead_len = 0;  // kRounds: the next unit's lengths, read a round ahead
      Unit ahead;
      bool more = kMany && place(0, ahead);
      if (more) {
        ahead_ctx = a.d.context_lens[ahead.r];
        ahead_len = tree_len(ahead.r);
      }
      int ks = 0, kph = 0;          // stage and phase of the next S
      int vs = 0, vph = 0, pk = 0;  // of the next P.V, and its tile's K stage
      auto next_k = [&]() {
        if (++ks == S::kKStages) {
          ks = 0;
          kph ^= 1;
        }
      };
      auto next_v = [&]() {
        if (++vs == S::kVStages) {
          vs = 0;
          vph ^= 1;
        }
        if (++pk == S::kKStages) pk = 0;
      };
      for (int round = 0; round < rounds && ok; ++round) {
        Unit w = unit0;
        if (kMany) {
          if (!more) break;
          w = ahead;
          measure(w, ahead_ctx, ahead_len);
          more = round + 1 < rounds && place(round + 1, ahead);
          if (more) {
            ahead_ctx = a.d.context_lens[ahead.r];
            ahead_len = tree_len(ahead.r);
          }
        }
        const int n_tiles = w.n_tiles;
        if (n_tiles <= 0) continue;
        if (t >= w.q_tiles) {  // a row tile without queries only gives the stages back
          for (int j = 0; j < n_tiles && ok; ++j) {
            ok = wait(&bars->k_full[ks], kph);
            if (ok) give_back(&bars->k_empty[ks]);
            ok = ok && wait(&bars->v_full[vs], vph);
            if (ok) give_back(&bars->v_empty[vs]);
            next_k();
            next_v();
          }
          continue;
        }
        const int qb = S::kQBufs == 2 ? units & 1 : 0;
        ok = wait(&bars->q_full[t][qb], (S::kQBufs == 2 ? units >> 1 : units) & 1);
        ++units;
        for (int j = 0; j < 2 && j < n_tiles && ok; ++j) {
          ok = wait(&bars->k_full[ks], kph);
          if (ok) issue_s((g + j) & 1, ks, qb);
          next_k();
        }
        for (int j = 0; j < n_tiles && ok; ++j, ++g) {
          const int buf = g & 1, ph = (g >> 1) & 1;
          ok = wait2(&bars->v_full[vs], vph, &bars->p_full[t][buf], ph);
          if (ok) {
            give_back(&bars->k_empty[pk]);  // the weights were made from S_j
            issue_pv(buf, vs, j == 0);
          }
          if (j + 2 < n_tiles) {
            ok = ok && wait2(&bars->k_full[ks], kph, &bars->o_done[t][buf], ph);
            if (ok) {
              give_back(&bars->v_empty[vs]);
              issue_s(buf, ks, qb);
            }
            next_k();
          }
          next_v();
        }
        // the last two tiles' V, once their products are done
        for (int back = kMany ? min(n_tiles, 2) : 0; back > 0 && ok; --back) {
          const uint32_t gt = g - back;
          const int st = vs >= back ? vs - back : vs - back + S::kVStages;
          ok = wait(&bars->o_done[t][gt & 1], (gt >> 1) & 1);
          if (ok) give_back(&bars->v_empty[st]);
        }
      }
      if (!ok && leader) report(a.d.err, PKV_DEVERR_TIMEOUT);
      __syncwarp();
    }
  } else {
    // ---------------------------- softmax ----------------------------
    set_max_regs_up<S::kSoftmaxRegs>();
    const int tid = threadIdx.x & 127;  // within the row tile
    const int qt = (warp >> 2) - 1;
    const int quad = warp & 3;  // TMEM sub-partition of this warp
    const int row = quad * 32 + lane;
    uint32_t g = 0;       // tiles of this row tile so far
    uint32_t v_tile = 0;  // tiles through the V ring so far
    int units = 0;        // of this row tile so far
    bool loaded = false;  // kTwoQ: the unit's queries are in their buffer
    // kRounds: the next two units, their lengths read that much ahead
    // (their places are worked out again: registers are dearer than that)
    int ahead_ctx = 0, ahead_len = 0, far_ctx = 0, far_len = 0;
    auto read_lengths = [&](int round, int& ctx, int& n_new) {
      Unit u;
      if (round < rounds && place(round, u)) {
        ctx = a.d.context_lens[u.r];
        n_new = tree_len(u.r);
      }
    };
    if constexpr (kMany) {
      read_lengths(0, ahead_ctx, ahead_len);
      read_lengths(1, far_ctx, far_len);
    }
    for (int round = 0; round < rounds; ++round) {
    Unit w = unit0;
    if (kMany) {
      if (!place(round, w)) break;
      measure(w, ahead_ctx, ahead_len);
      ahead_ctx = far_ctx;
      ahead_len = far_len;
      read_lengths(round + 2, far_ctx, far_len);
    }
    const int r = w.r, kvh = w.kvh, pos0 = w.pos0, ctx = w.ctx, n_new = w.n_new, base = w.base, n_pos = w.n_pos;
    const int first_block = w.first_block, key_end = w.key_end, n_tiles = w.n_tiles;
    const int qi = pos0 + qt * kPosPerTile + (row >> 2);  // query index
    const bool in_shape = qi < a.d.q_len;
    const bool row_valid = in_shape && qi < n_new;
    auto out_row = [&]() -> int64_t {
      return (static_cast<int64_t>(r) * a.d.q_len + qi) * hq + kvh * kGroup + (row & 3);
    };
    auto part_slot = [&]() -> int64_t { return out_row() * a.d.part_slots + split; };
    // zeros for a row without a result (padding, or nothing visible)
    auto write_empty = [&]() {
      if constexpr (kMode == MaskedMode::kWorkspace) {
        a.d.part_lse[part_slot()] = -INFINITY;
      } else if constexpr (kMode == MaskedMode::kCluster) {
        part_ml[qt * kRowsPerTile + row] = make_float2(-INFINITY, 0.f);
      } else {
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.d.out) + out_row() * kHeadDim);
#pragma unroll
        for (int c = 0; c < kHeadDim * 2 / 16; ++c) o[c] = make_uint4(0, 0, 0, 0);
      }
    };
    // first token of tile j of the split
    auto tile_token = [&](int j) -> int {
      const int i = t_first + j;
      return (i < w.sink_tiles ? i * S::kTileBlocks : first_block + (i - w.sink_tiles) * S::kTileBlocks) * kBlockSize;
    };
    if (n_tiles <= 0) {
      if (in_shape) write_empty();
      continue;
    }
    const bool tile_live = qt < w.q_tiles;
    if (kMany && !tile_live) {
      if (in_shape) write_empty();
      v_tile += n_tiles;
      continue;
    }
    // the unit before has left its results' way, its query buffer (all four warps)
    if constexpr (kMany) {
      if (units > 0) named_barrier_sync(1 + qt, 128);
    }
    const int qb = S::kQBufs == 2 ? units & 1 : 0;
    ++units;
    uint8_t* qarea = smem + S::kOffQ + (qb * kQTiles + qt) * kQTileBytes;  // queries, then results on their way out
    if (!loaded) {
      // this row tile's queries -> 128-byte swizzled K-major tile, two 64-dim
      // halves; thread t loads 16-byte chunk t % 16 of every (threads / 16)-th
      // row, eight loads in flight
      const int ch = tid & 15;
      const uint16_t* qbase = static_cast<const uint16_t*>(a.d.q);
      constexpr int kStep = 128 / 16;
      constexpr int kDeep = kMany ? 16 : 8;  // loads in flight (16: one trip, 8: fewer registers)
#pragma unroll
      for (int k0 = 0; k0 < kRowsPerTile / kStep; k0 += kDeep) {
        uint4 v[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          const int m = (tid >> 4) + kStep * (k0 + k);
          const int qim = pos0 + qt * kPosPerTile + (m >> 2);
          v[k] = make_uint4(0, 0, 0, 0);
          if (qim < n_new)
            v[k] = *reinterpret_cast<const uint4*>(
                qbase + ((static_cast<int64_t>(r) * a.d.q_len + qim) * hq + kvh * kGroup + (m & 3)) * kHeadDim + ch * 8);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          const int m = (tid >> 4) + kStep * (k0 + k);
          *reinterpret_cast<uint4*>(qarea + (ch >> 3) * kQHalfBytes + tc::sw128_offset(m, (ch & 7) * 8)) = v[k];
        }
      }
      tc::fence_proxy_async_smem();
      mbar_arrive(&bars->q_full[qt][qb]);
    }
    loaded = false;
    Unit next;
    if (kMany && !kTwoQ && round + 1 < rounds && place(round + 1, next)) {  // the next unit's queries towards L2
      const int qa = next.pos0 + qt * kPosPerTile + (row >> 2);
      if (qa < a.d.q_len) {
        const uint16_t* next_q =
            static_cast<const uint16_t*>(a.d.q) +
            ((static_cast<int64_t>(next.r) * a.d.q_len + qa) * hq + next.kvh * kGroup + (row & 3)) * kHeadDim;
        prefetch_l2(next_q);
        prefetch_l2(next_q + kHeadDim / 2);
      }
    }
    if constexpr (kTwoQ) {
      // The next unit's queries into the other buffer, if it has some here.
      // (Before the tiles: inside their loop it costs every tile 4 %.  With one
      // buffer, 4 x 1480 queries of window 90 take 93.5 us instead of 85.7.)
      Unit n;
      if (round + 1 < rounds && place(round + 1, n)) {
        measure(n, ahead_ctx, ahead_len);
        loaded = n.n_tiles > 0 && qt < n.q_tiles;
        if (loaded) {
          const uint16_t* qn = static_cast<const uint16_t*>(a.d.q) +
                               ((static_cast<int64_t>(n.r) * a.d.q_len + n.pos0 + qt * kPosPerTile) * hq +
                                n.kvh * kGroup) * kHeadDim;
          const uint32_t dst = smem_addr(smem + S::kOffQ + ((qb ^ 1) * kQTiles + qt) * kQTileBytes);
          const int ch = tid & 15, n_q = n.n_new - n.pos0 - qt * kPosPerTile;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int m = (tid >> 4) + 8 * k;
            const bool in = (m >> 2) < n_q;
            cp_async16(dst + (ch >> 3) * kQHalfBytes + tc::sw128_offset(m, (ch & 7) * 8),
                       qn + (in ? (static_cast<int64_t>(m >> 2) * hq + (m & 3)) * kHeadDim + ch * 8 : 0), in ? 16 : 0);
          }
        }
      }
    }
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tcol = tmem + lane_off + qt * S::kTileCols;
    const float c = a.d.scale_log2;  // > 0: the max of raw scores scales to the max of scaled ones
    const bool warp_live = pos0 + qt * kPosPerTile + quad * 8 < n_new;  // some row of the warp has a query
    // the keys a row sees in [tok, tok + 64), one bit per key
    const uint64_t* mrow = nullptr;
    uint64_t mask0 = 0, mask1 = 0;  // its first words, read before they are needed
    if constexpr (kMask == MaskKind::kTree) {
      mrow = a.tree_mask + (static_cast<int64_t>(r) * a.d.q_len + (row_valid ? qi : 0)) * a.mask_words;
      mask0 = mrow[0];
      if (a.mask_words > 1) mask1 = mrow[1];
    }
    auto mask_word = [&](int w) -> uint64_t {
      return w >= a.mask_words ? 0ull : (w == 0 ? mask0 : (w == 1 ? mask1 : mrow[w]));
    };
    // (in_sinks: the range belongs to a tile of sink blocks, whose places past
    // them are holes: the window's keys are read by the tiles after it)
    auto visible = [&](int tok, bool in_sinks) -> uint64_t {
      if constexpr (kMask == MaskKind::kTree) {
        const int d = base - tok;  // committed tokens of the range
        uint64_t m = low_bits(d);
        if (d < 64) {
          const int o = -d;  // draft at bit 0 (negative: drafts start at bit d)
          if (o < 0) {
            m |= mask0 << d;
          } else {
            const int w = o >> 6, sh = o & 63;
            m |= mask_word(w) >> sh;
            if (sh != 0) m |= mask_word(w + 1) << (64 - sh);
          }
        }
        return m & low_bits(key_end - tok);
      } else {
        const int p = base + qi;
        const int hi = p + 1 - tok;
        const uint64_t sinks = low_bits(min(a.num_sinks - tok, hi));
        return in_sinks ? sinks : sinks | (low_bits(hi) & ~low_bits(p - a.window + 1 - tok));
      }
    };
    // does some row of this CTA see the tile only in part?
    auto partial = [&](int tok) -> bool {
      if constexpr (kMask == MaskKind::kTree) return tok + S::kTileTokens > base;
      const int p_first = base + pos0, p_last = base + pos0 + n_pos - 1;
      return tok + S::kTileTokens - 1 > p_first ||
             !(tok > p_last - a.window || tok + S::kTileTokens <= a.num_sinks);
    };
    float m_stale = -INFINITY;  // scaled max the weights are taken against (lags the true max by < 2^16)
    float l = 0.f;              // the sum of the weights
    for (int j = 0; j < n_tiles && tile_live; ++j) {
      const int buf = (g + j) & 1, ph = ((g + j) >> 1) & 1;
      const int tok = tile_token(j);
      const uint32_t scol = tcol + buf * S::kTileTokens;
      // keep `ok` warp-uniform: the tcgen05 loads below are warp-collective
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[qt][buf], ph));
      if (!ok) break;
      const bool part = partial(tok);
      float s[64];  // raw scores of the tile's tokens
      if (warp_live) {
        tc::fence_after_sync();
        tc::tmem_ld32(scol, s);
        tc::tmem_ld32(scol + 32, s + 32);
        tc::tmem_wait_ld();
        if (__builtin_expect(part, 0)) {
          const uint64_t m = row_valid ? visible(tok, tok < first_block * kBlockSize) : 0ull;
          const uint32_t lo = static_cast<uint32_t>(m), hi = static_cast<uint32_t>(m >> 32);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (!(lo & (1u << e))) s[e] = -INFINITY;
            if (!(hi & (1u << e))) s[32 + e] = -INFINITY;
          }
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
        const bool grow = mx > m_stale + kRescaleThreshold;  // also true the first time a row sees a key
        const float m_new = grow ? mx : m_stale;
        const float alpha = grow ? exp2_approx(m_stale - m_new) : 1.f;  // 0 while m_stale is -inf
        if (__builtin_expect(__any_sync(0xffffffffu, grow && j > 0 && m_stale != -INFINITY), 0)) {
          // O holds weights taken against the old maxima: rescale this warp's rows
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_done[qt][buf ^ 1], ((g + j - 1) >> 1) & 1));
          tc::fence_after_sync();
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            float o[32];
            const uint32_t ocol = tcol + S::kColO + 32 * cc;
            tc::tmem_ld32(ocol, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tc::tmem_st32(ocol, o);
          }
          tc::tmem_wait_st();
        }
        l *= alpha;
        m_stale = m_new;
      }
      // V rows of the slots past the context (weight 0, but they may hold
      // anything): zero them
      if (__builtin_expect(part && ctx > tok && ctx < tok + S::kTileTokens && (ctx & (kBlockSize - 1)) != 0, 0)) {
        const int st = (v_tile + j) % S::kVStages;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->v_full[st], ((v_tile + j) / S::kVStages) & 1));
        uint8_t* vt = smem + S::kOffV + st * S::kStageBytes;
        const int t0 = ctx - tok, t1 = (t0 + kBlockSize - 1) & ~(kBlockSize - 1);
        for (int idx = tid; idx < (t1 - t0) * 16; idx += 128) {
          const int tk = t0 + (idx >> 4), ch = idx & 15;
          *reinterpret_cast<uint4*>(vt + (ch >> 3) * S::kHalfBytes + tk * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();  // before the MMA that the weights' arrival lets go
      }
      if (warp_live) {
        const float nm = (m_stale == -INFINITY) ? 0.f : -m_stale;
        const float2 c2 = make_float2(c, c);
        const float2 nm2 = make_float2(nm, nm);
        float2 acc2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // P_j overwrites the S_j buffer it came from, 2 BF16 per 32-bit column
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t pk[16], pr[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __ffma2_rn(make_float2(s[32 * cc + 2 * e], s[32 * cc + 2 * e + 1]), c2, nm2);
            const float p0 = exp2_approx(x.x);
            const float p1 = exp2_approx(x.y);
            acc2[e & 1] = __fadd2_rn(acc2[e & 1], make_float2(p0, p1));
            pk[e] = pack_bf16x2(p0, p1);
            if constexpr (S::kRemainder)
              pr[e] = pack_bf16x2(p0 - __uint_as_float(pk[e] << 16), p1 - __uint_as_float(pk[e] & 0xffff0000u));
          }
          tc::tmem_st16u(scol + 16 * cc, pk);
          if constexpr (S::kRemainder) tc::tmem_st16u(scol + 32 + 16 * cc, pr);
        }
        l += (acc2[0].x + acc2[0].y) + (acc2[1].x + acc2[1].y);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(&bars->p_full[qt][buf]);
    }
    if (kTwoQ && loaded) {
      cp_async_wait_all();
      tc::fence_proxy_async_smem();
      mbar_arrive(&bars->q_full[qt][qb ^ 1]);
    }
    v_tile += n_tiles;
    if (tile_live) g += n_tiles;
    // ---- epilogue ----
    // Results go through the row tile's query area (no product reads it any
    // more) so that the rows are written as whole 256-byte lines: a thread's
    // own row in 16-byte pieces costs 32 separate lines an instruction.
    if (ok && tile_live)
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_done[qt][(g - 1) & 1], ((g - 1) >> 1) & 1));
    if constexpr (kMode == MaskedMode::kCluster) {
      // the partials go over the rings: no row tile's products may still read them
      if constexpr (kQTiles == 2) named_barrier_sync(1, 128 * kQTiles);
    }
    if (tile_live && warp_live) {
      tc::fence_after_sync();
      const bool live = row_valid && l != 0.f && ok;  // (a NaN sum stays one)
      const float inv = live ? 1.f / l : 0.f;
      uint8_t* stage = qarea + quad * 32 * 256;  // this warp's 32 rows of 256 bytes
      // 16-byte chunk ch of row m sits at chunk ch ^ (m % 8): four wavefronts either way
      auto chunk = [&](int m, int ch) -> uint4* { return reinterpret_cast<uint4*>(stage + m * 256 + ((ch ^ (m & 7)) << 4)); };
      if constexpr (kMode == MaskedMode::kCluster) {
        // un-normalised FP32 row, 16-byte chunk ch at ch ^ (row % 8)
        const int m = qt * kRowsPerTile + row;
        uint8_t* po = smem + S::kOffPartO + m * kHeadDim * 4;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float o[32];
          tc::tmem_ld32(tcol + S::kColO + 32 * cc, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(po + (((8 * cc + e) ^ (row & 7)) << 4)) =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
        part_ml[m] = live ? make_float2(m_stale, l) : make_float2(-INFINITY, 0.f);
      } else if constexpr (kToOut) {
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float o[32];
          tc::tmem_ld32(tcol + S::kColO + 32 * cc, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) {
              w.x = pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv);
              w.y = pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv);
              w.z = pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv);
              w.w = pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv);
            }
            *chunk(lane, 4 * cc + e) = w;
          }
        }
        __syncwarp();
        // a position's four heads lie together: 1 KB, two stores of the warp
        const int q0 = pos0 + qt * kPosPerTile + quad * 8;  // the warp's first position
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.d.out) +
                                            ((static_cast<int64_t>(r) * a.d.q_len + q0) * hq + kvh * kGroup) * kHeadDim) +
                   lane;
        const int n_out = a.d.q_len - q0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int m = 2 * i + (lane >> 4), ch = lane & 15;
          if ((i >> 1) < n_out) o[(i & 1) * 32] = *chunk(m, ch);
          if (i & 1) o += hq * (kHeadDim / 8);
        }
      } else {
        // FP32 partials, 64 dims (256 bytes) of each row at a time
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            float o[32];
            tc::tmem_ld32(tcol + S::kColO + 64 * pass + 32 * cc, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(chunk(lane, 8 * cc + e)) =
                  make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int m = 2 * i + (lane >> 4), ch = lane & 15;
            const int mq = pos0 + qt * kPosPerTile + ((quad * 32 + m) >> 2);
            if (mq < n_new) {  // (a row that sees nothing is skipped by the combine kernel)
              const int64_t orow = (static_cast<int64_t>(r) * a.d.q_len + mq) * hq + kvh * kGroup + (m & 3);
              *reinterpret_cast<uint4*>(a.d.part_o + (orow * a.d.part_slots + split) * kHeadDim + 64 * pass + 4 * ch) =
                  *chunk(m, ch);
            }
          }
          if (pass == 0) __syncwarp();
        }
        if (in_shape) a.d.part_lse[part_slot()] = live ? (m_stale + log2f(l)) * kLn2 : -INFINITY;
      }
    } else if (in_shape) {
      write_empty();
    }
    }
    if (!ok && lane == 0) report(a.d.err, PKV_DEVERR_TIMEOUT);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, S::kTmemCols);
  }

  if constexpr (kMode == MaskedMode::kCluster) {
    // Each CTA merges its share of the rows (one per warp at a time, 4 dims a
    // lane) from every split's partial: O = sum_s 2^(m_s - m) O_s / sum_s
    // 2^(m_s - m) l_s.
    cluster_sync_all();
    const uint32_t splits = gridDim.y, rank = cluster_cta_rank();
    const Unit& w = unit0;
    const int rows = min(kPos, a.d.q_len - w.pos0) * kGroup;  // rows of the shape, padding included
    for (int m = static_cast<int>(rank) * S::kWarps + warp; m < rows; m += static_cast<int>(splits) * S::kWarps) {
      float ms[kMaxClusterSplits], ls[kMaxClusterSplits];
      float4 os[kMaxClusterSplits];
#pragma unroll
      for (int k = 0; k < kMaxClusterSplits; ++k) {
        ms[k] = -INFINITY;
        ls[k] = 0.f;
        if (k < static_cast<int>(splits)) {
          // its own partials first, then round the cluster: reads of one CTA's
          // memory by all at once would queue there
          const uint32_t src = rank + k < splits ? rank + k : rank + k - splits;
          const uint32_t ml = map_shared_to_rank(part_ml + m, src);
          ms[k] = ld_cluster_f32(ml);
          ls[k] = ld_cluster_f32(ml + 4);
          os[k] = ld_cluster_f32x4(map_shared_to_rank(smem + S::kOffPartO + m * kHeadDim * 4 + ((lane ^ (m & 7)) << 4), src));
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < kMaxClusterSplits; ++k) mx = fmaxf(mx, ms[k]);
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxClusterSplits; ++k) {
        // saw nothing: its O holds anything (a row whose scores are all NaN
        // leaves the maximum at -inf too, but its sum is NaN)
        if (ls[k] == 0.f) continue;
        const float w = exp2_approx(ms[k] - mx);
        sum = fmaf(ls[k], w, sum);
        o.x = fmaf(os[k].x, w, o.x);
        o.y = fmaf(os[k].y, w, o.y);
        o.z = fmaf(os[k].z, w, o.z);
        o.w = fmaf(os[k].w, w, o.w);
      }
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      uint2 packed;
      packed.x = pack_bf16x2(o.x * inv, o.y * inv);
      packed.y = pack_bf16x2(o.z * inv, o.w * inv);
      const int64_t mrow =
          (static_cast<int64_t>(w.r) * a.d.q_len + w.pos0 + (m >> 2)) * hq + w.kvh * kGroup + (m & 3);
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.d.out) + mrow * kHeadDim)[lane] = packed;
    }
    cluster_sync_all();  // a partial stays until every CTA has read it
  }
}

template <int kQTiles, MaskKind kMask, MaskedMode kMode>
__global__ void __launch_bounds__(ShapeOf<kQTiles, kMode>::kThreads, ShapeOf<kQTiles, kMode>::kCtasPerSm)
    paged_masked_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                           const MaskedArgs a) {
  paged_masked_tc_body<kQTiles, kMask, kMode>(k_map, v_map, a);
}

// Opt the kernel in to its dynamic shared memory, once per device.
template <int kQTiles, MaskKind kMask, MaskedMode kMode>
cudaError_t allow_smem(int* device) {
  static std::atomic<bool> done[64];  // per device; host threads may race on a first call
  cudaError_t e = cudaGetDevice(device);
  if (e != cudaSuccess) return e;
  if (*device < 0 || *device >= 64) return cudaErrorInvalidDevice;
  if (!done[*device]) {
    e = cudaFuncSetAttribute(paged_masked_tc_kernel<kQTiles, kMask, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ShapeOf<kQTiles, kMode>::kSmem);
    if (e != cudaSuccess) return e;
    done[*device] = true;
  }
  return cudaSuccess;
}

// Clusters of `splits` CTAs that are resident at once on device `dev` (the
// current one); 0 when that cannot be asked (no device).
template <int kQTiles>
int max_clusters(int splits, int dev) {
  static std::atomic<int> known[64][kMaxClusterSplits + 1];  // per device, + 1
  int n = known[dev][splits].load(std::memory_order_relaxed);
  if (n == 0) {
    if (allow_smem<kQTiles, MaskKind::kTree, MaskedMode::kCluster>(&dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1, static_cast<unsigned>(splits));
    cfg.blockDim = dim3(Shape<kQTiles>::kThreads);
    cfg.dynamicSmemBytes = Shape<kQTiles>::kSmem;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1;
    attr.val.clusterDim.y = static_cast<unsigned>(splits);
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, paged_masked_tc_kernel<kQTiles, MaskKind::kTree, MaskedMode::kCluster>, &cfg) !=
        cudaSuccess) {
      cudaGetLastError();
      c = 0;
    }
    n = c + 1;
    known[dev][splits].store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

template <int kQTiles, MaskKind kMask, MaskedMode kMode>
cudaError_t launch_variant(const CUtensorMap& kmap, const CUtensorMap& vmap, const MaskedArgs& a,
                           cudaStream_t stream) {
  using S = ShapeOf<kQTiles, kMode>;
  int dev = 0;
  const cudaError_t e = allow_smem<kQTiles, kMask, kMode>(&dev);
  if (e != cudaSuccess) return e;
  auto kernel = paged_masked_tc_kernel<kQTiles, kMask, kMode>;
  constexpr int kPos = kPosPerTile * kQTiles;
  int64_t x = static_cast<int64_t>(a.d.num_seqs) * a.d.num_kv_heads * ((a.d.q_len + kPos - 1) / kPos);
  if (kMode == MaskedMode::kRounds) x = std::min(x, static_cast<int64_t>(a.resident));
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(a.d.num_splits));
  return launch_pdl(kernel, grid, dim3(S::kThreads), S::kSmem, stream,
                    kMode == MaskedMode::kCluster ? static_cast<unsigned>(a.d.num_splits) : 1u, kmap, vmap, a);
}

template <int kQTiles, MaskKind kMask>
cudaError_t launch_mask(const CUtensorMap& kmap, const CUtensorMap& vmap, const MaskedArgs& a, cudaStream_t stream) {
  if (a.d.num_splits == 1 && a.rounds) return launch_variant<kQTiles, kMask, MaskedMode::kRounds>(kmap, vmap, a, stream);
  if (a.d.num_splits == 1) return launch_variant<kQTiles, kMask, MaskedMode::kDirect>(kmap, vmap, a, stream);
  if (a.d.part_o != nullptr) return launch_variant<kQTiles, kMask, MaskedMode::kWorkspace>(kmap, vmap, a, stream);
  if (a.d.num_splits > kMaxClusterSplits) return cudaErrorInvalidValue;
  return launch_variant<kQTiles, kMask, MaskedMode::kCluster>(kmap, vmap, a, stream);
}

template <int kQTiles>
cudaError_t launch_shape(const CUtensorMap& kmap, const CUtensorMap& vmap, const MaskedArgs& a, MaskKind mask,
                         cudaStream_t stream) {
  return mask == MaskKind::kTree ? launch_mask<kQTiles, MaskKind::kTree>(kmap, vmap, a, stream)
                                 : launch_mask<kQTiles, MaskKind::kWindow>(kmap, vmap, a, stream);
}

}  // namespace

int masked_positions_per_cta(bool wide) { return wide ? 2 * kPosPerTile : kPosPerTile; }
int masked_ctas_per_sm(bool wide) { return wide ? Shape<2>::kCtasPerSm : Shape<1>::kCtasPerSm; }

int masked_max_clusters(bool wide, int splits, int device) {
  return wide ? max_clusters<2>(splits, device) : max_clusters<1>(splits, device);
}

cudaError_t launch_paged_masked_tc(const MaskedArgs& a, MaskKind mask, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.d.num_blocks) * a.d.num_kv_heads * kBlockSize;
  if (rows + kBlockSize >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
  CUtensorMap kmap, vmap;
  if (!make_pool_map(&kmap, a.d.k_cache, rows) || !make_pool_map(&vmap, a.d.v_cache, rows)) return cudaErrorInvalidValue;
  return a.wide ? launch_shape<2>(kmap, vmap, a, mask, stream)
                                  : launch_shape<1>(kmap, vmap, a, mask, stream);
}

}  // namespace pkv
