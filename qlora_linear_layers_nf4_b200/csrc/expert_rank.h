// Host interface of the expert layer's rank-r activations (expert_rank.cu).
#pragma once

#include <cuda.h>

#include "kernels.h"

namespace nf4 {

enum RankKind { kRankT = 0, kRankU };

struct RankParams {
  RankKind kind;
  int red_steps;     // 64-deep steps of the reduction
  int NP, r;         // columns, rounded up to 64 and kept
  int slices, tmem_cols;
  int E, M;
  int f16;
  float scale;       // s
  float lo_mul;      // scale of a term over the one before
  const int32_t* offsets;
  uint16_t* out[3];  // T, or the terms of U; null past the last
  uint32_t* status;
  int* zero;         // ints cleared on the way (for the kernel after), or null
  int zero_n;
};

// One product, prepared on the host before the first launch of a call.
struct ExpertRank {
  CUtensorMap ma, mb;
  RankParams p;
  dim3 grid;
  size_t smem = 0;
  bool prepare(const GroupedArgs& g, RankKind kind, void* out0, void* out1, void* out2, int sms);
  cudaError_t run(cudaStream_t st, int* launches) const;
};

}  // namespace nf4
