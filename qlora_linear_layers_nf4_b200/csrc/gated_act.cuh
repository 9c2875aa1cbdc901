// The gate's activation and its derivative.  Both forms are g times a logistic function:
//   SiLU              act(g) = g q,  q = 1 / (1 + exp(-g))
//   GELU, tanh form   act(g) = g q,  q = 1 / (1 + exp(-y)),  y = 2 sqrt(2 / pi) (g + 0.044715 g^3)
// (0.5 (1 + tanh z) is the logistic function of 2 z), so with y = g for SiLU
//   act'(g) = q + g q (1 - q) y'(g).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace nf4 {
namespace gated {

constexpr int kSilu = 0;       // nf4_activation
constexpr int kGeluTanh = 1;

// FAST: exp and reciprocal of a few units in the last place (the exponent's rounding makes
// |y| 2^-24 of q), for results that are rounded to 16 bits or, in the gradients, summed over
// rows beside errors as large; else the rounded functions (fp32 mode).  Results below 2^-126
// count as 0.
template <bool FAST>
__device__ __forceinline__ float logistic(float y) {
  if (!FAST) return 1.0f / (1.0f + expf(-y));
  float e, q;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.0f + e));
  return q;
}

constexpr float kGeluTwoC = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// Within -64 .. 64 (a NaN stays one): past it q is 0 or 1 whatever g is, and g^3 stays finite.
__device__ __forceinline__ float within_64(float g) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(g), "f"(-64.0f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(c), "f"(64.0f));
  return c;
}

template <bool FAST>
__device__ __forceinline__ float act(int kind, float g) {
  if (kind == kSilu) return g * logistic<FAST>(g);
  const float c = within_64(g);
  return g * logistic<FAST>(kGeluTwoC * fmaf(kGeluCubic * c * c, c, c));
}

struct ActGrad {
  float a, d;   // act(g), act'(g)
};
template <bool FAST>
__device__ __forceinline__ ActGrad act_grad(int kind, float g) {
  if (kind == kSilu) {
    const float q = logistic<FAST>(g);
    return ActGrad{g * q, fmaf(q * (1.0f - q), g, q)};
  }
  const float c = within_64(g), c2 = kGeluCubic * c * c;
  const float q = logistic<FAST>(kGeluTwoC * fmaf(c2, c, c));
  return ActGrad{g * q, fmaf(q * (1.0f - q), c * kGeluTwoC * fmaf(3.0f, c2, 1.0f), q)};
}

// Two fp32 values in one register pair: one instruction does both.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split2(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 both(float x) { return f2(x, x); }

// act(g) and act'(g) of two values, as act_grad<true>.
template <int KIND>
__device__ __forceinline__ void act_grad2(F2 g, F2* a, F2* d) {
  F2 y, slope;
  if (KIND == kSilu) {
    y = mul2(g, both(-1.4426950408889634f));
    slope = g;
  } else {
    const float2 s = split2(g);
    const F2 c = f2(within_64(s.x), within_64(s.y));
    const F2 c2 = mul2(mul2(c, both(kGeluCubic)), c);
    y = mul2(fma2(c2, c, c), both(kGeluTwoC * -1.4426950408889634f));
    slope = mul2(mul2(c, both(kGeluTwoC)), fma2(c2, both(3.0f), both(1.0f)));
  }
  float2 e = split2(y), q;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.x) : "f"(1.0f + e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.y) : "f"(1.0f + e.y));
  const F2 q2 = f2(q.x, q.y);
  *a = mul2(g, q2);
  *d = fma2(mul2(q2, fma2(q2, both(-1.0f), both(1.0f))), slope, q2);
}

}  // namespace gated
}  // namespace nf4
