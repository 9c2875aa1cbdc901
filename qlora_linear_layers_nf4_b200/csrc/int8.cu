// 8-bit integers with a scale per row: the quantizer and the linear layer.
//
// Quantize: scale = fp32(max |x| / 127), code = the integer nearest to
// x / scale, ties to even.  The quotient is taken exactly without a division
// per element: q = rint(x * (1 / scale)) is at most one off, and the remainder
// x - q scale, which one FMA gives exactly (it has at most 24 bits), says
// whether a neighbour is nearer.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "expert_gemm.h"
#include "kernels.h"
#include "nf4_common.cuh"
#include "tc_common.cuh"

namespace nf4 {
namespace {

using namespace tc;

// ------------------------------------------------------------------ quantize

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  __device__ static float one(const float* p) { return *p; }
  __device__ static void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  __device__ static float one(const __half* p) { return __half2float(*p); }
  __device__ static void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
};

struct RowScale {
  float s, inv;
  bool zero;    // codes are 0: the scale is 0 or NaN
  bool tiny;    // subnormal scale: 1 / s may overflow, divide instead
};

__device__ __forceinline__ RowScale row_scale(uint32_t top_bits) {
  RowScale r;
  r.s = top_bits >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                                : __fdiv_rn(__uint_as_float(top_bits), 127.0f);
  r.zero = !(r.s > 0.0f);
  r.tiny = r.s < 1.17549435e-38f;
  r.inv = __fdiv_rn(1.0f, r.s);
  return r;
}

__device__ __forceinline__ int int8_code(float x, const RowScale& r) {
  if (r.zero) return 0;
  float q = rintf(r.tiny ? __fdiv_rn(x, r.s) : __fmul_rn(x, r.inv));
  const float rem = fmaf(-q, r.s, x);
  const float d = 2.0f * fabsf(rem);
  int c = int(q);
  if (d > r.s || (d == r.s && (c & 1))) c += rem > 0.0f ? 1 : -1;
  return min(max(c, -127), 127);
}

constexpr int kQThreads = 256;
constexpr int kQKeep = 4;        // 16-byte vectors of a row that a thread keeps in registers

// One CTA per row.  VEC: rows start on 16-byte boundaries (and the codes on
// vector boundaries).  The row is read once: what fits stays in registers
// between the maximum and the codes, the rest is read again from L2.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads) int8_quantize_kernel(const T* __restrict__ x, int cols,
                                                                 int8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
  constexpr int V = Elem<T>::kVec;
  grid_dep_wait();
  const int64_t row = blockIdx.x;
  const T* xr = x + row * cols;
  int8_t* cr = codes + row * cols;
  const int t = threadIdx.x;
  uint32_t top = 0;
  uint4 keep[kQKeep];
  const int nvec = VEC ? cols / V : 0;
  if (VEC) {
    const uint4* xv = reinterpret_cast<const uint4*>(xr);
#pragma unroll
    for (int i = 0; i < kQKeep; ++i) {
      const int at = t + i * kQThreads;
      keep[i] = at < nvec ? __ldg(xv + at) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kQKeep; ++i) {
      float f[V];
      Elem<T>::unpack(keep[i], f);
#pragma unroll
      for (int u = 0; u < V; ++u) top = max(top, __float_as_uint(f[u]) & 0x7fffffffu);
    }
    for (int at = t + kQKeep * kQThreads; at < nvec; at += kQThreads) {
      float f[V];
      Elem<T>::unpack(__ldg(xv + at), f);
#pragma unroll
      for (int u = 0; u < V; ++u) top = max(top, __float_as_uint(f[u]) & 0x7fffffffu);
    }
  } else {
    for (int at = t; at < cols; at += kQThreads)
      top = max(top, __float_as_uint(Elem<T>::one(xr + at)) & 0x7fffffffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  __shared__ uint32_t part[kQThreads / 32];
  if ((t & 31) == 0) part[t >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQThreads / 32; ++w) top = max(top, part[w]);
  const RowScale r = row_scale(top);
  if (t == 0) scales[row] = r.s;
  if (VEC) {
    const uint4* xv = reinterpret_cast<const uint4*>(xr);
    auto put = [&](int at, const uint4& v) {
      float f[V];
      Elem<T>::unpack(v, f);
      uint32_t w[V / 4];
#pragma unroll
      for (int g = 0; g < V / 4; ++g) {
        w[g] = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) w[g] |= (uint32_t(int8_code(f[4 * g + u], r)) & 0xffu) << (8 * u);
      }
      if (V == 4) *reinterpret_cast<uint32_t*>(cr + int64_t(at) * V) = w[0];
      else *reinterpret_cast<uint2*>(cr + int64_t(at) * V) = make_uint2(w[0], w[V / 4 - 1]);
    };
#pragma unroll
    for (int i = 0; i < kQKeep; ++i) {
      const int at = t + i * kQThreads;
      if (at < nvec) put(at, keep[i]);
    }
    for (int at = t + kQKeep * kQThreads; at < nvec; at += kQThreads) put(at, __ldg(xv + at));
  } else {
    for (int at = t; at < cols; at += kQThreads) cr[at] = int8_t(int8_code(Elem<T>::one(xr + at), r));
  }
}

template <typename T>
cudaError_t quantize_t(const void* x, int64_t rows, int64_t cols, int8_t* codes, float* scales, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(rows), 1, 1);
  cfg.blockDim = dim3(kQThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = prof_on() ? 0 : 1;
  const T* xt = static_cast<const T*>(x);
  return cols % Elem<T>::kVec == 0
             ? cudaLaunchKernelEx(&cfg, int8_quantize_kernel<T, true>, xt, int(cols), codes, scales)
             : cudaLaunchKernelEx(&cfg, int8_quantize_kernel<T, false>, xt, int(cols), codes, scales);
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int in_dtype, int64_t rows, int64_t cols, int8_t* codes,
                                 float* scales, int sms, cudaStream_t st, int* launches) {
  (void)sms;
  NF4_PROF_BEGIN(st, kKInt8Quantize);
  cudaError_t e = in_dtype == NF4_F32   ? quantize_t<float>(x, rows, cols, codes, scales, st)
                  : in_dtype == NF4_F16 ? quantize_t<__half>(x, rows, cols, codes, scales, st)
                                        : quantize_t<__nv_bfloat16>(x, rows, cols, codes, scales, st);
  NF4_PROF_END(st, kKInt8Quantize);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_int8_linear(const Int8LinearArgs& a, int sms, cudaStream_t st, int* launches) {
  return launch_int8_gemm(a, sms, st, launches);
}

}  // namespace nf4
