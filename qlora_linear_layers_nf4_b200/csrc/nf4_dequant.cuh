// NF4 codes to 16-bit values in registers and in the 128-byte-swizzled tiles
// that the tensor core reads (the expert GEMM).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nf4_common.cuh"
#include "tc_common.cuh"

namespace nf4 {

namespace expert {

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
// Two values rounded (nearest, ties to even) to the compute type: f16 or bf16.
__device__ __forceinline__ uint32_t pack2(bool f16, float lo, float hi) {
  return f16 ? f16x2_rn(lo, hi) : bf16x2_rn(lo, hi);
}
__device__ __forceinline__ float2 unpack2(bool f16, uint32_t w) {
  return f16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
             : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// The sixteen dequantized values of one block, bf16(L[c] * scale) (or f16)
// with the fp32 product rounded to nearest even, split into byte planes so a
// lookup is a register byte-permute: lo[q] holds the low bytes of entries
// 4q..4q+3, hi[q] their high bytes.
struct BlockTable {
  uint32_t lo[4];
  uint32_t hi[4];
};

__device__ __forceinline__ BlockTable make_table(float scale, bool f16) {
  uint32_t p[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j] = pack2(f16, __fmul_rn(__uint_as_float(level_bits(2 * j)), scale),
                 __fmul_rn(__uint_as_float(level_bits(2 * j + 1)), scale));
  }
  BlockTable t;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    t.lo[q] = prmt(p[2 * q], p[2 * q + 1], 0x6420u);
    t.hi[q] = prmt(p[2 * q], p[2 * q + 1], 0x7531u);
  }
  return t;
}

// Four codes (the low 16 bits of `w`: two packed bytes, even element in the
// high nibble) -> four bf16 values as two bf16x2 words in element order.
__device__ __forceinline__ uint2 decode4(uint32_t w, const BlockTable& t) {
  const uint32_t sel = w & 0x7777u;                          // code & 7 per nibble
  const uint32_t pick = ((w >> 1) & 0x4444u) | 0x3210u;      // code >= 8 -> upper plane
  const uint32_t lo = prmt(prmt(t.lo[0], t.lo[1], sel), prmt(t.lo[2], t.lo[3], sel), pick);
  const uint32_t hi = prmt(prmt(t.hi[0], t.hi[1], sel), prmt(t.hi[2], t.hi[3], sel), pick);
  // lo/hi bytes are in nibble order (odd element first within a byte).
  return make_uint2(prmt(lo, hi, 0x4051u), prmt(lo, hi, 0x6273u));
}

// Half a block (32 elements, 16 code bytes at `codes`, smem) into 16-byte
// chunks 4*half .. 4*half+3 of row `row` of a 128-byte-swizzled bf16 tile.
__device__ __forceinline__ void dequant_half_row(const uint8_t* codes, float scale, uint8_t* tile,
                                                 uint32_t row, uint32_t half, bool f16) {
  const uint4 c = *reinterpret_cast<const uint4*>(codes);
  const BlockTable t = make_table(scale, f16);
  const uint32_t words[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint2 a = decode4(words[k], t);
    const uint2 b = decode4(words[k] >> 16, t);
    *reinterpret_cast<uint4*>(tile + tc::sw128_offset(row, 4 * half + k)) = make_uint4(a.x, a.y, b.x, b.y);
  }
}

__device__ __forceinline__ float load_scale(const uint8_t* absmax_q, const float* absmax,
                                            float s_g, bool dq, int64_t idx) {
  return dq ? __fmul_rn(float(__ldg(absmax_q + idx)), s_g) : __ldg(absmax + idx);
}

}  // namespace expert
}  // namespace nf4
