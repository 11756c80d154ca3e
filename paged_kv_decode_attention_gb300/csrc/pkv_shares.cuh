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
  constexpr int kFlight = 4;  // rows of a lane, neighbours: their reads are in flight together
  auto cost = [&](int tiles) -> int { return tiles > 0 ? tiles + job_cost : 0; };
  auto read = [&](int r0, int (&x)[kFlight]) -> int {
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int r = r0 + kFlight * lane + k;
      x[k] = r < rows ? tiles_of(r) : 0;
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) sum += cost(x[k]);
    return sum;
  };
  // (Loops stay rolled: a warp runs this once, from a cold instruction cache.)
  int x[kFlight];
  int sum = read(0, x);  // costs of the lane's rows, once for each KV head
  int all = sum;
#pragma unroll 1
  for (int r0 = 32 * kFlight; r0 < rows; r0 += 32 * kFlight) {
    int y[kFlight];
    all += read(r0, y);
  }
  const uint32_t total = __reduce_add_sync(0xffffffffu, all) * num_kv_heads;
  const uint32_t grid = gridDim.x;
  Share s{};
  s.per = max(static_cast<int>((total + grid - 1) / grid), min_share);
  const int t0 = s.per * static_cast<int>(blockIdx.x);
  s.left = min(s.per, static_cast<int>(total) - t0);
  if (s.left <= 0) return s;
  int before = 0;
#pragma unroll 1
  for (int r0 = 0;; r0 += 32 * kFlight) {
    if (r0 > 0) sum = read(r0, x);
    const int mine = sum * num_kv_heads;
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > t0);
    if (past == 0) {
      before += __shfl_sync(0xffffffffu, upto, 31);
      continue;
    }
    const int at = __ffs(past) - 1;
    int start = before + __shfl_sync(0xffffffffu, upto - mine, at);
    bool found = false;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int tiles = __shfl_sync(0xffffffffu, x[k], at);
      const int c = cost(tiles) * num_kv_heads;
      if (!found && t0 < start + c) {
        found = true;
        s.tiles = tiles;
        s.row = r0 + kFlight * at + k;
      }
      if (!found) start += c;
    }
    const uint32_t c = cost(s.tiles);
    s.kvh = static_cast<uint32_t>(t0 - start) / c;
    s.into = (t0 - start) - s.kvh * static_cast<int>(c);
    return s;
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
