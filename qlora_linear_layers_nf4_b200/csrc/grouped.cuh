// Rows sorted by expert: the table that every kernel of the expert (grouped)
// linear builds in shared memory from the offsets in device memory, so that
// no row count ever travels to the host.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "nf4_common.cuh"

namespace nf4 {

// start[e] .. start[e + 1]: rows of expert e; tiles[e] .. tiles[e + 1]: its
// row tiles among those of all experts.
struct GroupTable {
  int start[kMaxExperts + 1];
  int tiles[kMaxExperts + 1];
};

// Fill the table (one whole warp).  Offsets are clamped to [0, M] and to the
// running maximum, so the groups never overlap or leave the matrix whatever
// the caller's memory holds; a clamped offset is recorded in *status.  An
// expert's rows are cut into ceil(rows / tile) tiles.
__device__ __forceinline__ void build_groups(GroupTable* t, const int32_t* __restrict__ offsets, int E,
                                             int M, int tile, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  int carry = 0;        // largest offset so far
  bool bad = false;
  for (int b = 0; b <= E; b += 32) {
    const int i = b + lane;
    const int raw = i <= E ? __ldg(offsets + i) : 0;
    int v = i <= E ? min(max(raw, 0), M) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    v = max(v, carry);
    if (i <= E) {
      t->start[i] = v;
      bad |= v != raw;
    }
    carry = __shfl_sync(0xffffffffu, v, 31);
  }
  __syncwarp();
  int sum = 0;
  for (int b = 0; b < E; b += 32) {
    const int i = b + lane;
    const int mine = i < E ? (t->start[i + 1] - t->start[i] + tile - 1) / tile : 0;
    int v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (i < E) t->tiles[i] = sum + v - mine;
    sum += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) t->tiles[E] = sum;
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(status, NF4_ERR_INVALID_ARG);
  __syncwarp();
}

// Expert of row tile `tile` (< tiles[E]): the last e with tiles[e] <= tile,
// which has rows because tiles[e + 1] > tile.
__device__ __forceinline__ int expert_of_tile(const GroupTable* t, int E, int tile) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t->tiles[mid] <= tile) lo = mid; else hi = mid;
  }
  return lo;
}

// Most row tiles that M rows of E experts can make: sum ceil(c / tile).
inline int64_t max_row_tiles(int64_t M, int64_t E, int64_t tile) {
  return M / tile + (E < M ? E : M);
}

}  // namespace nf4
