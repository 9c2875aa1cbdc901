// Host interface of the gated layer's weight-streaming forward (gated_decode.cu).
#pragma once

#include <cuda.h>

#include "gated.h"

namespace nf4 {

struct GatedDecodeParams {
  int M, N, K, r;
  int n_tiles, k_chunks;    // tiles of 64 outputs, 256-wide chunks of a row
  int row_tiles;            // groups of tokens
  int whole;                // tiles that a CTA has of its own, behind
  int rest, rest_ctas;      // the first tiles, which rest_ctas CTAs share
  int bs_shift, dq, act;
  int vec_scales;           // a row's four scales of a chunk are one aligned vector
  const uint8_t* absmax_q[2];
  const float* absmax[2];
  const float* absmax_scale[2];
  const uint16_t* B;        // [2][N][r]
  const uint16_t* T;        // [2][M][r]
  const uint16_t* bias;     // [2][N] or null
  uint16_t* h;
  uint16_t* pre;            // [2][M][N] or null
  float* partials;          // [CTA][2][16][128]: a share's split tiles
  int* counters;            // [CTA]: CTAs that have written a split tile's part, by its first CTA
  uint32_t* status;
};

size_t gated_decode_scratch_bytes();

struct GatedDecode {
  CUtensorMap codes[2], x;
  GatedDecodeParams p;
  unsigned grid = 0;
  int np = 16;              // tokens per group
  bool f16 = false;
  // T: written by the kernel launched just before, which also clears the counters
  bool prepare(const GatedArgs& a, const void* T, uint8_t* scratch, int sms);
  cudaError_t run(cudaStream_t st, int* launches) const;
};

// T of a few tokens; clears the decode kernel's counters, if there are any.
cudaError_t launch_gated_t_small(const GatedArgs& a, void* T, int* counters, cudaStream_t st, int* launches);

}  // namespace nf4
