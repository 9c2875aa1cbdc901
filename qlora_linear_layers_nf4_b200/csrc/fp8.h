// The 8-bit floating point linear: arguments of a call, and its tensor-core product.
#pragma once

#include <cuda.h>

#include "fp8_plan.h"
#include "kernels.h"

namespace nf4 {

struct Fp8LinearArgs {
  const uint8_t* w;        // [N, K] e4m3
  const float* w_scale;    // [ceil(N / 128), ceil(K / 128)]
  int64_t M, N, K;
  const uint8_t* x;        // [M, K] e4m3
  const float* x_scale;    // [M, ceil(K / 128)]
  int dtype;               // of y and bias
  const void* bias;
  void* y;
  uint32_t* status;
};

cudaError_t launch_fp8_quantize(const void* x, int in_dtype, int64_t rows, int64_t cols, int block_rows, uint8_t* codes,
                                float* scales, int sms, cudaStream_t stream, int* launches);
cudaError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols, int block_rows,
                                  int out_dtype, void* out, int sms, cudaStream_t stream, int* launches);
// x: [M, K] of a.dtype, quantized into codes and scales on the way, or (x_scale given) e4m3;
// a.x and a.x_scale are set here.
cudaError_t launch_fp8_linear(const Fp8LinearArgs& a, const void* x, const float* x_scale, uint8_t* codes,
                              float* scales, int sms, cudaStream_t stream, int* launches);

struct Fp8Params {
  int M, N;
  int kb;                  // blocks of 128 along K
  int row_tiles, tiles;
  uint32_t x_bytes;        // of a CTA's tokens in a stage
  int dtype;
  const float* w_scale;
  const float* x_scale;
  const void* bias;
  void* y;
  uint32_t* status;
};

// The product on the tensor cores (fp8_gemm.cu), prepared on the host before the first
// launch of a call.
struct Fp8Gemm {
  CUtensorMap mx, mw, my;
  Fp8Params p;
  unsigned grid = 0;
  int tile_n = 0;          // as in Fp8GemmPlan
  int parts = 1;
  bool prepare(const Fp8LinearArgs& a, int sms);
  cudaError_t run(cudaStream_t st, int* launches) const;
};

}  // namespace nf4
