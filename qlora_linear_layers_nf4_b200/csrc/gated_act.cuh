// The gate's activation and its derivative.  Both forms are g times a logistic function:
//   SiLU              act(g) = g q,  q = 1 / (1 + exp(-g))
//   GELU, tanh form   act(g) = g q,  q = 1 / (1 + exp(-y)),  y = 2 sqrt(2 / pi) (g + 0.044715 g^3)
// (0.5 (1 + tanh z) is the logistic function of 2 z), so with y = g for SiLU
//   act'(g) = q + g q (1 - q) y'(g).
#pragma once

#include <cuda_runtime.h>

namespace nf4 {
namespace gated {

constexpr int kSilu = 0;       // nf4_activation
constexpr int kGeluTanh = 1;

// FAST: exp and reciprocal of a few units in the last place (below |g| = 20, q is off by
// less than 2^-20 of itself), for results that are rounded to 16 bits or, in the gradients,
// summed over rows beside errors as large; else the rounded functions (fp32 mode).
template <bool FAST>
__device__ __forceinline__ float logistic(float y) {
  return FAST ? __fdividef(1.0f, 1.0f + __expf(-y)) : 1.0f / (1.0f + expf(-y));
}

constexpr float kGeluTwoC = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

template <bool FAST>
__device__ __forceinline__ float act(int kind, float g) {
  const float y = kind == kSilu ? g : kGeluTwoC * fmaf(kGeluCubic * g * g, g, g);
  return g * logistic<FAST>(y);
}

struct ActGrad {
  float a, d;   // act(g), act'(g)
};
template <bool FAST>
__device__ __forceinline__ ActGrad act_grad(int kind, float g) {
  const float g2 = kGeluCubic * g * g;
  const float y = kind == kSilu ? g : kGeluTwoC * fmaf(g2, g, g);
  const float slope = kind == kSilu ? 1.0f : kGeluTwoC * fmaf(3.0f, g2, 1.0f);
  const float q = logistic<FAST>(y);
  const float p = q * (1.0f - q);
  // where q is 0 or 1 the second term is 0, though g times the slope may be infinite
  return ActGrad{g * q, p > 0.0f ? fmaf(p, g * slope, q) : q};
}

}  // namespace gated
}  // namespace nf4
