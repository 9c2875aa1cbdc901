// Host interface of the expert GEMM (expert_gemm.cu).
#pragma once

#include <cuda.h>

#include "kernels.h"

namespace nf4 {

struct ExpertMaps {
  CUtensorMap tok_l, tok_s;   // tokens: 128-row and 32-row boxes
  CUtensorMap ad_l, ad_s;     // T or U: the same
  CUtensorMap wad;            // adapter operand on the weight side
  CUtensorMap w;              // kI8: the weight
};

struct ExpertParams {
  int M, E;
  int out_cols;               // outputs of an expert: N (kFwd, kI8) or K (kDx)
  int w_rows, w_cols;         // N, K of an expert
  int r;
  int main_steps, adapter_steps;
  int col_tiles;
  int block_chunks_shift, dq;   // log2 of the 64-element chunks per block
  int out_dtype;              // kI8: nf4_dtype of out and bias
  const int32_t* offsets;     // null: all M rows are the one expert's
  const uint8_t* codes;
  int codes32;                // codes start on a 32-byte boundary
  const uint8_t* absmax_q;
  const float* absmax;
  const float* absmax_scale;
  const void* bias;
  void* out;
  const float* w_scale;       // kI8
  const float* x_scale;       // kI8
  uint32_t* status;
};

// y or dx of a stack of experts, prepared on the host (tensor maps encoded)
// before the first launch of a call.  `ad`: T (forward) or U (backward),
// [M, r] in the compute type, written by the kernel launched just before.
struct ExpertGemm {
  ExpertMaps maps;
  ExpertParams p;
  unsigned grid = 0;
  int parts = 1;              // MMAs of 256 tokens a tile
  bool dx = false, f16 = false;
  bool prepare(const GroupedArgs& g, bool backward, const void* ad, int sms);
  cudaError_t run(cudaStream_t st, int* launches) const;
};

// The 8-bit linear on the tensor cores.
struct Int8Gemm {
  ExpertGemm g;
  bool prepare(const Int8LinearArgs& a, int sms);
  cudaError_t run(cudaStream_t st, int* launches) const;
};

}  // namespace nf4
