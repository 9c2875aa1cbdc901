// 8-bit integers with a scale per row: the quantizer and the linear layer.
//
// Quantize: scale = fp32(max |x| / 127), code = the integer nearest to
// x / scale, ties to even.  The quotient is taken exactly without a division
// per element: q = rint(x * (1 / scale)) is at most one off, and the remainder
// x - q scale, which one FMA gives exactly (it has at most 24 bits), says
// whether a neighbour is nearer.  Rounding to an integer is the addition of 1.5
// 2^23, whose low byte then is the code: the conversion instructions run at an
// eighth of that rate and bounded the kernel.
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

// Four codes, packed.  The common case is four operations an element; a group in
// which one remainder reaches half a step (or whose scale is 0, NaN or subnormal)
// takes int8_code for all four.
__device__ __forceinline__ uint32_t int8_codes4(const float* x, const RowScale& r) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
  const float half = 0.5f * r.s;
  bool rare = r.zero || r.tiny;
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float m = fmaf(x[i], r.inv, kMagic);
    b[i] = __float_as_uint(m);
    const float rem = fmaf(kMagic - m, r.s, x[i]);
    rare |= !(fabsf(rem) < half);
  }
  if (rare) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = uint32_t(int8_code(x[i], r));
  }
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
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
    // unsigned: the column after the last may lie past 2^31
    for (uint32_t at = t; at < uint32_t(cols); at += kQThreads)
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
      for (int g = 0; g < V / 4; ++g) w[g] = int8_codes4(f + 4 * g, r);
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
    for (uint32_t at = t; at < uint32_t(cols); at += kQThreads) cr[at] = int8_t(int8_code(Elem<T>::one(xr + at), r));
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

// ------------------------------------------------------------------ linear, few tokens

// y for up to four tokens: the weight bytes are the whole cost, and one launch
// the largest other one, so the tokens are quantized here too.  A CTA holds the
// codes of all tokens in shared memory (every CTA makes them again: 2 M K bytes
// from L2 against a kernel of its own) and 32 weight rows, two to a warp, whose
// first 4 KB are already on their way while the tokens are quantized.  Sums by
// dp4a, exact; the warp's lanes meet in one integer reduction a sum.
constexpr int kSmThreads = 512;
constexpr int kSmRows = 2;                             // weight rows per warp
constexpr int kSmTileRows = kSmRows * kSmThreads / 32;
constexpr int kSmAhead = 4;                            // 16-byte loads a lane has in flight per row
constexpr int64_t kSmMaxCodes = 160 * 1024;            // M * K

template <typename T, int MT>
__global__ void __launch_bounds__(kSmThreads) int8_small_kernel(const Int8LinearArgs a, const T* __restrict__ x,
                                                               const float* __restrict__ given_scale) {
  extern __shared__ __align__(16) int8_t codes[];      // [M][K]
  __shared__ float scale[MT];
  __shared__ uint32_t part[kSmThreads / 32];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int K = int(a.K), M = int(a.M);
  const int vecs = K / 16;
  grid_dep_wait();
  const int64_t n0 = int64_t(blockIdx.x) * kSmTileRows + warp * kSmRows;
  const uint4* w[kSmRows];
#pragma unroll
  for (int i = 0; i < kSmRows; ++i) w[i] = reinterpret_cast<const uint4*>(a.w + (n0 + i < a.N ? n0 + i : a.N - 1) * a.K);
  uint4 wv[kSmRows][kSmAhead];
  auto load_w = [&](int v0) {
#pragma unroll
    for (int j = 0; j < kSmAhead; ++j)
#pragma unroll
      for (int i = 0; i < kSmRows; ++i) {
        const int v = v0 + 32 * j + lane;
        wv[i][j] = v < vecs ? __ldg(w[i] + v) : make_uint4(0u, 0u, 0u, 0u);
      }
  };
  load_w(0);

  if constexpr (sizeof(T) == 1) {
    for (int i = t; i < M * vecs; i += kSmThreads)
      reinterpret_cast<uint4*>(codes)[i] = __ldg(reinterpret_cast<const uint4*>(x) + i);
    if (t < M) scale[t] = given_scale[t];
  } else {
    constexpr int V = Elem<T>::kVec;
    for (int m = 0; m < M; ++m) {
      const uint4* xv = reinterpret_cast<const uint4*>(x + int64_t(m) * K);
      uint32_t top = 0;
      for (int i = t; i < K / V; i += kSmThreads) {
        float f[V];
        Elem<T>::unpack(__ldg(xv + i), f);
#pragma unroll
        for (int u = 0; u < V; ++u) top = max(top, __float_as_uint(f[u]) & 0x7fffffffu);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) part[warp] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kSmThreads / 32; ++i) top = max(top, part[i]);
      const RowScale r = row_scale(top);
      if (t == 0) scale[m] = r.s;
      for (int i = t; i < K / V; i += kSmThreads) {
        float f[V];
        Elem<T>::unpack(__ldg(xv + i), f);
#pragma unroll
        for (int g = 0; g < V / 4; ++g)
          reinterpret_cast<uint32_t*>(codes)[(m * K + i * V) / 4 + g] = int8_codes4(f + 4 * g, r);
      }
      __syncthreads();   // part may be written again
    }
  }
  __syncthreads();

  int acc[kSmRows][MT];
#pragma unroll
  for (int i = 0; i < kSmRows; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = 0;
  for (int v0 = 0; v0 < vecs; v0 += 32 * kSmAhead) {
#pragma unroll
    for (int j = 0; j < kSmAhead; ++j) {
      const int v = v0 + 32 * j + lane;
      if (v < vecs) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (m >= M) break;
          const uint4 c = *reinterpret_cast<const uint4*>(codes + m * K + v * 16);
#pragma unroll
          for (int i = 0; i < kSmRows; ++i) {
            int s = acc[i][m];
            s = __dp4a(int(wv[i][j].x), int(c.x), s);
            s = __dp4a(int(wv[i][j].y), int(c.y), s);
            s = __dp4a(int(wv[i][j].z), int(c.z), s);
            acc[i][m] = __dp4a(int(wv[i][j].w), int(c.w), s);
          }
        }
      }
    }
    if (v0 + 32 * kSmAhead < vecs) load_w(v0 + 32 * kSmAhead);
  }
#pragma unroll
  for (int i = 0; i < kSmRows; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m >= M) break;
      const int sum = __reduce_add_sync(0xffffffffu, acc[i][m]);
      const int64_t n = n0 + i;
      if (lane == m && n < a.N) {
        float v = __fmul_rn(__fmul_rn(float(sum), scale[m]), a.w_scale[n]);
        const int64_t at = int64_t(m) * a.N + n;
        if (a.dtype == NF4_F32) {
          if (a.bias != nullptr) v = __fadd_rn(v, static_cast<const float*>(a.bias)[n]);
          static_cast<float*>(a.y)[at] = v;
        } else if (a.dtype == NF4_F16) {
          if (a.bias != nullptr) v = __fadd_rn(v, __half2float(static_cast<const __half*>(a.bias)[n]));
          static_cast<__half*>(a.y)[at] = __float2half_rn(v);
        } else {
          if (a.bias != nullptr) v = __fadd_rn(v, __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[n]));
          static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
        }
      }
    }
}

template <typename T, int MT>
cudaError_t small_tm(const Int8LinearArgs& a, const void* x, const float* scale, cudaStream_t st) {
  static PerDeviceOnce attr_done;
  const int dev = PerDeviceOnce::current();
  if (!attr_done.done(dev)) {
    const cudaError_t e = cudaFuncSetAttribute(int8_small_kernel<T, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmMaxCodes));
    if (e != cudaSuccess) return e;
    attr_done.mark(dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.N + kSmTileRows - 1) / kSmTileRows), 1, 1);
  cfg.blockDim = dim3(kSmThreads, 1, 1);
  cfg.dynamicSmemBytes = size_t(a.M * a.K);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = prof_on() ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, int8_small_kernel<T, MT>, a, static_cast<const T*>(x), scale);
}
template <typename T>
cudaError_t small_t(const Int8LinearArgs& a, const void* x, const float* scale, cudaStream_t st) {
  return a.M == 1 ? small_tm<T, 1>(a, x, scale, st) : a.M == 2 ? small_tm<T, 2>(a, x, scale, st)
                  : small_tm<T, 4>(a, x, scale, st);
}

// Its products cost dp4a's on every SM; the GEMM's cost nothing beside its fixed 8 to
// 12 us.  Measured, this kernel against the GEMM, us: 4096 x 4096 with 1, 2, 4 and 8
// tokens 4.9, 6.9, 9.5 and 16 against 12; 8192 x 4096 with 2 and 4 tokens 8.6 and 13.5
// against 12.5; 11008 x 16384 with 1 and 2 tokens 37 and 42 against 39.
bool use_small(const Int8LinearArgs& a) {
  return a.M * a.K <= kSmMaxCodes && (a.M == 1 || (a.M <= 4 && a.M * a.N * a.K <= int64_t(100) << 20));
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

cudaError_t launch_int8_linear(const Int8LinearArgs& given, const void* x, const float* x_scale, int8_t* codes,
                               float* scales, int sms, cudaStream_t st, int* launches) {
  Int8LinearArgs a = given;
  if (use_small(a)) {
    NF4_PROF_BEGIN(st, kKInt8Linear);
    cudaError_t e = x_scale != nullptr      ? small_t<int8_t>(a, x, x_scale, st)
                    : a.dtype == NF4_F32    ? small_t<float>(a, x, nullptr, st)
                    : a.dtype == NF4_F16    ? small_t<__half>(a, x, nullptr, st)
                                            : small_t<__nv_bfloat16>(a, x, nullptr, st);
    NF4_PROF_END(st, kKInt8Linear);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) ++*launches;
    return e;
  }
  Int8Gemm g;
  a.x = x_scale != nullptr ? static_cast<const int8_t*>(x) : codes;
  a.x_scale = x_scale != nullptr ? x_scale : scales;
  if (!g.prepare(a, sms)) return cudaErrorInvalidValue;
  if (x_scale == nullptr) {
    const cudaError_t e = launch_int8_quantize(x, a.dtype, a.M, a.K, codes, scales, sms, st, launches);
    if (e != cudaSuccess) return e;
  }
  return g.run(st, launches);
}

}  // namespace nf4
