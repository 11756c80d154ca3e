// pkv_shares.cuh -- work cut by tiles, not by requests.  A call's rows (a
// request's, or a row tile's of it) times its KV heads are jobs of some tiles
// each; all jobs in a row, each counted as its tiles and `job_cost` more for
// its start and end, are divided evenly among the CTAs of the grid, whatever
// the rows' lengths are.  A job that a share's end cuts leaves partials, at most
// two per CTA (the first job's end and the last one's start), which a second
// kernel joins.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "pkv_kernels.h"

namespace pkv {

// Where a CTA's share starts.
struct Share {
  int row, kvh;  // the job
  int tiles;     // its tiles
  int into;      // how far into its cost the share starts
  int left;      // cost of the share (<= 0: none)
  int per;       // cost of every share but the last
};

// Warp-collective.  tiles_of(row): tiles of one job of the row, 0 = no job.  (The
// host has seen to it that all costs together fit into 31 bits.)
template <typename TilesOf>
__device__ __forceinline__ Share find_share(int rows, int num_kv_heads, int job_cost, int min_share, int lane,
                                            TilesOf tiles_of) {
  constexpr int kFlight = 4;  // reads in flight: their latency is what this costs
  auto cost = [&](int tiles) -> int { return tiles > 0 ? tiles + job_cost : 0; };
  auto read = [&](int r0, int* x) {
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int r = r0 + 32 * k + lane;
      x[k] = r < rows ? tiles_of(r) : 0;
    }
  };
  int first[kFlight], total = 0;
  read(0, first);
#pragma unroll
  for (int k = 0; k < kFlight; ++k) total += cost(first[k]);
  for (int r0 = 32 * kFlight; r0 < rows; r0 += 32 * kFlight) {
    int x[kFlight];
    read(r0, x);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) total += cost(x[k]);
  }
  total = __reduce_add_sync(0xffffffffu, total) * num_kv_heads;
  const int grid = gridDim.x;
  Share s{};
  s.per = max((total + grid - 1) / grid, min_share);
  const int t0 = s.per * static_cast<int>(blockIdx.x);
  s.left = min(s.per, total - t0);
  if (s.left <= 0) return s;
  int before = 0;
  for (int r0 = 0;; r0 += 32 * kFlight) {
    int x[kFlight];
    if (r0 == 0) {
#pragma unroll
      for (int k = 0; k < kFlight; ++k) x[k] = first[k];
    } else {
      read(r0, x);
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      int upto = cost(x[k]) * num_kv_heads;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + upto > t0);
      if (past != 0) {
        const int at = __ffs(past) - 1;
        s.tiles = __shfl_sync(0xffffffffu, x[k], at);
        const int start = before + __shfl_sync(0xffffffffu, upto, at) - cost(s.tiles) * num_kv_heads;
        s.row = r0 + 32 * k + at;
        s.kvh = (t0 - start) / cost(s.tiles);
        s.into = (t0 - start) - s.kvh * cost(s.tiles);
        return s;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
}

// What a share holds of the job that it is in: the tiles [begin, begin + take)
// (take 0: it ends before the job's first one).  The share then moves on.
__device__ __forceinline__ void take_of_job(int tiles, int job_cost, int& into, int& left, int& begin, int& take) {
  const int end = min(into + left, tiles + job_cost);
  begin = max(into - job_cost, 0);
  take = max(end - job_cost, 0) - begin;
  left -= end - into;
  into = 0;
}

}  // namespace pkv
