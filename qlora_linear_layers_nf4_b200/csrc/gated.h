// The gated feed-forward layer: arguments of a call, and the launches its files prepare.
#pragma once

#include <cuda.h>

#include "gated_plan.h"
#include "kernels.h"

namespace nf4 {

// p = 0: gate, p = 1: up, in every array of two.
struct GatedArgs {
  const nf4_weight* w[2];  // same rows (N), cols (K), block size and scale form
  int64_t M, N, K;
  int r;
  float s;                 // alpha / r
  int f16, f32;            // compute type (else bf16)
  int act;                 // nf4_activation
  const void* x;           // [M, K]
  const void* A;           // [2, r, K]
  const void* B;           // [2, N, r]
  const void* bias;        // [2, N] or null
  const void* dh;          // [M, N] (backward)
  const void* pre_in;      // [2, M, N] (backward): g, u
  const void* t_in;        // [2, M, r] or null (backward)
  void* h;                 // [M, N]
  void* pre_out;           // [2, M, N] or null
  void* t_out;             // [2, M, r] or null
  float* dA;               // [2, r, K]
  float* dB;               // [2, N, r]
  void* dx;                // [M, K] or null
  uint8_t* ws;
  uint32_t* status;
};

size_t gated_workspace_bytes(bool backward, bool f32, int64_t M, int64_t N, int64_t K, int r);
cudaError_t launch_gated_fwd(const GatedArgs& a, int sms, cudaStream_t stream, int* launches);
cudaError_t launch_gated_bwd(const GatedArgs& a, int sms, cudaStream_t stream, int* launches);

// The F32 compute dtype, on the CUDA cores (gated_simt.cu).
size_t gated_f32_workspace_bytes(bool backward, int64_t M, int64_t N, int r);
cudaError_t launch_gated_fwd_f32(const GatedArgs& a, int sms, cudaStream_t stream, int* launches);
cudaError_t launch_gated_bwd_f32(const GatedArgs& a, int sms, cudaStream_t stream, int* launches);

// ---- gated_gemm.cu

struct GatedMaps {
  CUtensorMap tok_l, tok_s;   // tokens, 128-row and 32-row boxes: x, or dg and du [2][M][N]
  CUtensorMap ad_l, ad_s;     // T or U [2][M][r]: the same
  CUtensorMap wad;            // backward: A [2][r][K]
  CUtensorMap codes[2];       // backward: NF4 codes
  CUtensorMap h, pre;         // forward: the results, in pieces of 32 tokens x 64 outputs
};

struct GatedParams {
  int M;
  int out_cols;               // N (forward) or K (backward)
  int w_rows, w_cols;         // N, K
  int r;
  int half_steps;             // steps of 64 of one projection: forward K / 64, backward ceil(N / 64)
  int main_steps;             // half_steps, or both projections' (backward)
  int ad_steps;               // ceil(r / 64), of one projection
  int col_tiles, row_tiles, tile_rows;
  int block_chunks_shift, dq; // log2 of the 64-element chunks per block
  int act;
  int codes32[2];             // codes start on a 32-byte boundary
  const uint8_t* codes[2];
  const uint8_t* absmax_q[2];
  const float* absmax[2];
  const float* absmax_scale[2];
  const void* B;              // forward: [2][N][r]
  const void* bias;
  void* out;                  // h or dx
  void* pre;                  // forward: [2][M][N] or null
  int splits;                 // of the reduction
  float* partials;            // of several splits: [split][M][2][N] or [split][M][K]
  uint32_t* status;
};

// h (and g, u) or dx, prepared on the host before the first launch of a call.  `ad`: T
// [2][M][r], or the terms of U [2][terms][M][r], of which the first are read; `tok`: x, or dg
// and du [2][M][N]; the kernels launched before write them.  `scratch`: gated_split_bytes.
struct GatedGemm {
  GatedMaps maps;
  GatedParams p;
  unsigned grid = 0;
  int parts = 1;              // MMAs of 256 tokens a tile
  bool dx = false, f16 = false;
  bool prepare(const GatedArgs& a, bool backward, const void* tok, const void* ad, void* scratch, int sms);
  cudaError_t run(cudaStream_t st, int* launches) const;
  cudaError_t sum(cudaStream_t st, int* launches) const;   // adds up the splits, if there are several
};

}  // namespace nf4
