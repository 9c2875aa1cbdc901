// NF4 codes to 16-bit values in registers (the expert GEMM and decode kernel).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nf4_common.cuh"

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

// Four codes given by their selectors (low 16 bits: the code's low three bits per
// nibble, and 4 * its top bit + the nibble's place) -> four 16-bit values as two
// words in element order.  Byte permutes and logic share one half-rate pipe,
// which is what bounds the GEMM, so both selectors are made for eight codes at
// a time.
__device__ __forceinline__ uint2 decode4(uint32_t sel, uint32_t pick, const BlockTable& t) {
  const uint32_t lo = prmt(prmt(t.lo[0], t.lo[1], sel), prmt(t.lo[2], t.lo[3], sel), pick);
  const uint32_t hi = prmt(prmt(t.hi[0], t.hi[1], sel), prmt(t.hi[2], t.hi[3], sel), pick);
  // lo/hi bytes are in nibble order (odd element first within a byte).
  return make_uint2(prmt(lo, hi, 0x4051u), prmt(lo, hi, 0x6273u));
}

// The codes of one 64-element chunk, 32 bytes of global memory that nothing
// writes meanwhile: one 32-byte load where they are so aligned.
struct Codes {
  uint32_t w[8];
};
__device__ __forceinline__ Codes load_codes64(const uint8_t* p, bool aligned32) {
  Codes c;
  if (aligned32) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3]), "=r"(c.w[4]), "=r"(c.w[5]), "=r"(c.w[6]), "=r"(c.w[7])
        : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    c = Codes{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  return c;
}

// The eight values of a word of codes.  (The shifts as high products, on the multiply
// pipe instead, were slower: 604 us against 594 in the GEMM, 100 against 96 in the
// decode kernel.)
__device__ __forceinline__ uint4 decode8(uint32_t w, const BlockTable& t) {
  const uint32_t sel = w & 0x77777777u;
  const uint32_t pick = ((w >> 1) & 0x44444444u) | 0x32103210u;
  const uint2 a = decode4(sel, pick, t);
  const uint2 b = decode4(sel >> 16, pick >> 16, t);
  return make_uint4(a.x, a.y, b.x, b.y);
}

// A row's 64 values, as eight 16-byte chunks of 16-bit values.
__device__ __forceinline__ void decode_row(const Codes& c, const BlockTable& t, uint4 (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = decode8(c.w[k], t);
}

}  // namespace expert
}  // namespace nf4
