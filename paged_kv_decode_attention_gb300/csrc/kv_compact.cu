// kv_compact.cu -- after a tree of drafted tokens has been verified, bring the
// accepted path's K and V together: new[base + j] = old[base + accepted[j]]
// for every layer and KV head, base = the committed tokens before the drafts
// ("Chapter 8: Inference Optimization" (clxhxhhr.top/posts/4341), §8.5.2:
// drafted positions are verified in one step and a part of them is kept;
// §8.3.1: every token's place is found through the block table).
//
// accepted rises (a parent is drafted before its children), so
// accepted[j] >= j and row j is written only after every row that reads it
// has been: a thread moves the same 16-byte piece of one row after another in
// rising order, a few at a time (all loads of a batch before its stores), and
// no two threads touch the same piece.  Rows that are in place already are
// skipped, neither read nor written.
//
// What bounds it: two accesses per moved byte and, for few rows, the chain
// lengths -> accepted -> block table -> row -> store.  One CTA per (request,
// layer): the chain is walked once for K and V and all heads, by the lanes of
// one warp, and the layers run side by side in one launch.
//
// Measured (q8_0, 36 layers x 128 requests, up to 8 of 61 drafts accepted):
// 11.8 us with the rows in L2, 19 us from HBM, where it reads 50 MB for 33 MB
// of rows: a row's scales are 8 bytes, a DRAM access brings 64.  One thread
// per piece, the scales beside the codes, in equal passes of at most 192
// threads (up to 320: 12.8 us in L2; always 128 with the scales after the
// codes: 12.4 and 20.4, and 7.0 instead of 5.2 with one KV head); 8 rows in
// flight instead of 4: 13.8 and 19.2.  CTAs that stay and let one warp walk
// ahead took 25 and 30 us, several layers per CTA with the loads of one before
// the stores of another 14 to 26 and 20 to 31: the many small CTAs hide the
// chain better.  One request alone: 2.6 us.
#include "pkv_common.cuh"
#include "pkv_kernels.h"

namespace pkv {
namespace {

constexpr int kMaxThreads = 192;
constexpr int kBatch = 4;  // rows in flight per thread

struct Move {
  int32_t src_blk, dst_blk;
  int16_t src_off, dst_off;
};

// Bytes of a slot's row inside a tile: pieces of 16 bytes, then (q8_0) 8 bytes of scales.
template <int kFormat>
struct RowShape {
  static constexpr int kTile = kFormat == PKV_KV_BF16 ? kTileBytes : (kFormat == PKV_KV_Q8_0 ? kQ8TileBytes : kFp8TileBytes);
  static constexpr int kRow = kFormat == PKV_KV_BF16 ? kHeadDim * 2 : kHeadDim;
  static constexpr int kPieces = kRow / 16;
};

template <typename T>
__device__ __forceinline__ void move_piece(uint8_t* pool, const Move* moves, int n, int64_t head_off,
                                           int64_t block_bytes, int base_off, int row_bytes) {
  for (int m0 = 0; m0 < n; m0 += kBatch) {
    T v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (m0 + u < n) {
        const Move mv = moves[m0 + u];
        v[u] = *reinterpret_cast<const T*>(pool + mv.src_blk * block_bytes + head_off + base_off + mv.src_off * row_bytes);
      }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (m0 + u < n) {
        const Move mv = moves[m0 + u];
        *reinterpret_cast<T*>(pool + mv.dst_blk * block_bytes + head_off + base_off + mv.dst_off * row_bytes) = v[u];
      }
  }
}

template <int kFormat>
__global__ void __launch_bounds__(kMaxThreads) kv_compact_kernel(const __grid_constant__ CompactArgs a) {
  using R = RowShape<kFormat>;
  extern __shared__ Move moves[];  // [max_accepted]
  __shared__ int s_moves;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  const int layer = blockIdx.y;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const int ctx = a.context_lens[r];
    const int n = a.tree_lens != nullptr ? a.tree_lens[r] : a.tree_len;
    const int m = a.num_accepted[r];
    const int32_t* acc = a.accepted + static_cast<int64_t>(r) * a.max_accepted;
    const int32_t* table = a.block_tables + static_cast<int64_t>(r) * a.max_blocks;
    unsigned int bad = 0;
    if (m < 0 || m > a.max_accepted || n < 0 || n > a.tree_len || m > n) bad = PKV_DEVERR_ACCEPTED;
    else if (m > 0 && (ctx < n || ctx > a.max_blocks * kBlockSize)) bad = PKV_DEVERR_CONTEXT;
    const int base = ctx - n;
    int count = 0;
    for (int j0 = 0; j0 < m && bad == 0; j0 += 32) {
      const int j = j0 + lane;
      int i = j;
      bool moved = false;
      Move mv{};
      if (j < m) {
        i = acc[j];
        const int before = j > 0 ? acc[j - 1] : -1;
        if (i <= before || i >= n) bad = PKV_DEVERR_ACCEPTED;
        moved = bad == 0 && i != j;
        if (moved) {
          const int s = base + i, d = base + j;
          mv.src_blk = table[s / kBlockSize];
          mv.dst_blk = table[d / kBlockSize];
          mv.src_off = static_cast<int16_t>(s % kBlockSize);
          mv.dst_off = static_cast<int16_t>(d % kBlockSize);
          if (mv.src_blk < 0 || mv.src_blk >= a.num_blocks || mv.dst_blk < 0 || mv.dst_blk >= a.num_blocks)
            bad = PKV_DEVERR_BLOCK_ID;
        }
      }
      const unsigned who = __ballot_sync(0xffffffffu, moved);
      if (moved) moves[count + __popc(who & ((1u << lane) - 1u))] = mv;
      count += __popc(who);
      bad = __reduce_or_sync(0xffffffffu, bad);
    }
    if (lane == 0) {
      if (bad != 0) report(a.err, bad);
      s_moves = bad != 0 ? 0 : count;  // a bad request is left as it is
    }
  }
  __syncthreads();
  const int n = s_moves;
  if (n == 0) return;
  const int64_t block_bytes = static_cast<int64_t>(a.num_kv_heads) * R::kTile;
  const int per_pool = a.num_kv_heads * R::kPieces;
  // pieces of 16 bytes, then (q8_0) the 8 bytes of scales of each head
  const int total = 2 * per_pool + (kFormat == PKV_KV_Q8_0 ? 2 * a.num_kv_heads : 0);
  for (int idx = threadIdx.x; idx < total; idx += blockDim.x) {
    if (idx < 2 * per_pool) {
      const int which = idx >= per_pool;
      const int p = idx - which * per_pool;
      const int h = p / R::kPieces;
      uint8_t* pool = static_cast<uint8_t*>(which ? a.v_caches[layer] : a.k_caches[layer]);
      move_piece<uint4>(pool, moves, n, static_cast<int64_t>(h) * R::kTile, block_bytes, (p - h * R::kPieces) * 16, R::kRow);
    } else {
      const int which = idx - 2 * per_pool >= a.num_kv_heads;
      const int h = idx - 2 * per_pool - which * a.num_kv_heads;
      uint8_t* pool = static_cast<uint8_t*>(which ? a.v_caches[layer] : a.k_caches[layer]);
      move_piece<uint2>(pool, moves, n, static_cast<int64_t>(h) * R::kTile, block_bytes, kQ8CodeBytes, 8);
    }
  }
}

template <int kFormat>
cudaError_t launch_format(const CompactArgs& a, int32_t num_seqs, int32_t layers, cudaStream_t stream) {
  // as many threads as a row of K and V has pieces, in equal passes
  using R = RowShape<kFormat>;
  const int items = 2 * a.num_kv_heads * (R::kPieces + (kFormat == PKV_KV_Q8_0 ? 1 : 0));
  const int passes = (items + kMaxThreads - 1) / kMaxThreads;
  const unsigned threads = static_cast<unsigned>(((items + passes - 1) / passes + 31) / 32 * 32);
  return launch_pdl(kv_compact_kernel<kFormat>, dim3(static_cast<unsigned>(num_seqs), static_cast<unsigned>(layers)),
                    dim3(threads), a.max_accepted * sizeof(Move), stream, 1, a);
}

}  // namespace

cudaError_t launch_kv_compact(const CompactArgs& a, int32_t num_seqs, int32_t layers, int32_t kv_format,
                              cudaStream_t stream) {
  static_assert(kMaxTree * sizeof(Move) <= 40 * 1024, "the list of moves fits in shared memory");
  switch (kv_format) {
    case PKV_KV_BF16: return launch_format<PKV_KV_BF16>(a, num_seqs, layers, stream);
    case PKV_KV_Q8_0: return launch_format<PKV_KV_Q8_0>(a, num_seqs, layers, stream);
    case PKV_KV_FP8_E4M3: return launch_format<PKV_KV_FP8_E4M3>(a, num_seqs, layers, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pkv
