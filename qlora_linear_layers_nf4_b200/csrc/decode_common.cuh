// What the weight-streaming kernels (expert, gated) share: MMAs on registers, 16-bit
// conversions, the lookup of a byte of codes.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace nf4 {
namespace decode {

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

template <bool F16>
__device__ __forceinline__ float2 two_floats(uint32_t w) {
  return F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
             : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <bool F16>
__device__ __forceinline__ uint32_t two_rounded(float lo, float hi) {
  if (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool F16>
__device__ __forceinline__ uint16_t one_rounded(float v) {
  return uint16_t(two_rounded<F16>(v, 0.0f) & 0xffffu);
}
template <bool F16>
__device__ __forceinline__ float one_float(uint16_t v) {
  return two_floats<F16>(uint32_t(v)).x;
}

// Two weights: byte J of `word` looked up in the lane's copy of the table, times
// the scale, rounded to the compute type.
template <int J, bool F16>
__device__ __forceinline__ uint32_t two_weights(const uint8_t* lut, uint32_t word, uint32_t lane8, float scale) {
  uint32_t at;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(at) : "r"(word), "r"(lane8), "n"(0x5504 | (J << 4)));   // {lane8.b0, word.bJ, 0, 0}
  uint64_t l = *reinterpret_cast<const uint64_t*>(lut + at), s2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(scale));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(l) : "l"(s2));
  return two_rounded<F16>(__uint_as_float(uint32_t(l)), __uint_as_float(uint32_t(l >> 32)));
}

// Eight products of two 16-byte chunks of 16-bit values, added to acc in order.
template <bool F16>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = two_floats<F16>(aw[i]), v = two_floats<F16>(bw[i]);
    acc = fmaf(u.x, v.x, acc);
    acc = fmaf(u.y, v.y, acc);
  }
  return acc;
}

}  // namespace decode
}  // namespace nf4
