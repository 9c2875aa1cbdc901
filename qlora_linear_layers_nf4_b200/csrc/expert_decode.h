// Host interface of the expert layer's weight-streaming forward (expert_decode.cu).
#pragma once

#include <cuda.h>

#include "kernels.h"

namespace nf4 {

constexpr int kDecodeMaxCtas = 160;   // most CTAs of a launch; sizes the scratch

struct DecodeParams {
  int M, E, N, K, r;
  int n_tiles, k_chunks;    // 128-row tiles of an expert, 256-wide chunks of a row
  int bs_shift, dq;
  int vec_scales;           // a row's four scales of a chunk are one aligned vector
  const int32_t* offsets;
  const uint8_t* absmax_q;
  const float* absmax;
  const float* absmax_scale;
  const uint16_t* B;
  const uint16_t* T;
  const uint16_t* bias;
  uint16_t* y;
  float* partials;          // [CTA][2][16][128]: a share's split tiles
  int* counters;            // [CTA]: CTAs that have written a split tile's part, by its first CTA
  uint32_t* status;
};

size_t decode_scratch_bytes();

struct ExpertDecode {
  CUtensorMap codes, x;
  DecodeParams p;
  unsigned grid = 0;
  int np = 16;              // tokens per row group
  bool f16 = false;
  // T: [M, r], written by the kernel launched just before, which also clears the counters
  bool prepare(const GroupedArgs& g, const void* T, uint8_t* scratch, int sms);
  cudaError_t run(cudaStream_t st, int* launches) const;
};

cudaError_t launch_expert_t_small(const GroupedArgs& g, void* T, int* counters, cudaStream_t st, int* launches);

}  // namespace nf4
