// Host interface of the expert layer's rank-r products (expert_rank.cu).
#pragma once

#include <cuda.h>

#include "kernels.h"

namespace nf4 {

enum RankKind { kRankT = 0, kRankU, kRankDB, kRankDA };

struct RankParams {
  RankKind kind;
  int Mo;            // gradients: output rows of an expert (N or K)
  int row_tiles;     // gradients: 128-row tiles of an expert
  int red_steps;     // rows: 64-deep steps of the reduction
  int NP, r;         // columns, rounded up to 64 and kept
  int slices, stages, tmem_cols;
  int E, M;
  int f16;
  float scale;       // s (T, U)
  float lo_mul, lo_scale;   // scale of U's second term and its inverse
  const int32_t* offsets;
  void* out;         // T, U (16-bit) or dB, dA (fp32)
  void* out_lo;      // U: the second term
  uint32_t* status;
  int* zero;         // ints cleared on the way (for the kernel after), or null
  int zero_n;
};

// One product, prepared on the host before the first launch of a call.
struct ExpertRank {
  CUtensorMap ma, mb, mb2;
  RankParams p;
  dim3 grid;
  size_t smem = 0;
  // in16, in16_lo: T (dB) or U's two terms (dA)
  bool prepare(const GroupedArgs& g, RankKind kind, const void* in16, const void* in16_lo, void* out, void* out_lo);
  // pdl: as a programmatic dependent of the kernel before on the stream
  cudaError_t run(cudaStream_t st, int* launches, bool pdl) const;
};

}  // namespace nf4
