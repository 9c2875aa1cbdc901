// Host interface of the expert layer's adapter gradients (expert_grad.cu).
#pragma once

#include <cuda.h>

#include "kernels.h"

namespace nf4 {

constexpr float kULoMul = 2048.0f;   // f16: scale of U's second term

struct GradMaps {
  CUtensorMap a[2];      // x, dy
  CUtensorMap b[2];      // the terms of U, T
};

struct GradJob {
  int Mo;                // outputs of an expert: K (dA) or N (dB)
  int row_tiles, tiles;
  int terms;
  int whole;             // Mo is a multiple of 64
  float* out;
};

struct GradParams {
  GradJob job[2];        // dA, dB
  int E, M, r;
  int col_tiles;
  int f16;
  int stages;
  uint32_t stage_bytes;
  float lo_scale;
  const int32_t* offsets;
  uint32_t* status;
};

// Both gradients, prepared on the host before the first launch of a call.
struct ExpertGrad {
  GradMaps maps;
  GradParams p;
  unsigned grid = 0;
  size_t smem = 0;
  // U: its terms one after another, [u_terms][M][r]
  bool prepare(const GroupedArgs& g, const void* T, const void* U, int u_terms, int sms);
  cudaError_t run(cudaStream_t st, int* launches) const;
};

}  // namespace nf4
