// 8-bit floating point (e4m3) with a scale for each block of 128: the quantizer, its
// inverse, and the linear layer for few tokens.
//
// A block is 128 columns of one row (activations: one scale a token and 128 channels) or of
// 128 rows (weights).  scale = fp32(max |x| / 448), code = the e4m3 value nearest to
// v = fp32(x / scale), ties to even; both quotients IEEE fp32 divisions, so the codes do not
// depend on which kernel made them.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fp8.h"
#include "nf4_common.cuh"
#include "tc_common.cuh"

namespace nf4 {
namespace {

using namespace tc;

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  __device__ static float one(const float* p) { return __ldg(p); }
  __device__ static void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  // The bits of the largest magnitude: of the vector's and `top` in the type's own form
  // (16-bit types two at a time), and that as a float's.
  __device__ static uint32_t larger(const uint4& v, uint32_t top) {
    top = __vimax3_u32(v.x & 0x7fffffffu, v.y & 0x7fffffffu, top);
    return __vimax3_u32(v.z & 0x7fffffffu, v.w & 0x7fffffffu, top);
  }
  __device__ static uint32_t as_float(uint32_t top) { return top; }
};
// Of 16-bit types.
__device__ __forceinline__ uint32_t larger2(const uint4& v, uint32_t top) {
  top = __vimax3_u16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, top);
  return __vimax3_u16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu, top);
}
__device__ __forceinline__ uint32_t halves_max(uint32_t top) { return max(top & 0xffffu, top >> 16); }
template <>
struct Elem<__nv_bfloat16> {
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static uint32_t larger(const uint4& v, uint32_t top) { return larger2(v, top); }
  __device__ static uint32_t as_float(uint32_t top) { return halves_max(top) << 16; }
};
template <>
struct Elem<__half> {
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
  __device__ static uint32_t larger(const uint4& v, uint32_t top) { return larger2(v, top); }
  __device__ static uint32_t as_float(uint32_t top) {
    return __float_as_uint(__half2float(__ushort_as_half(uint16_t(halves_max(top)))));
  }
};
template <typename T>
constexpr int kVec = 16 / int(sizeof(T));   // elements of a 16-byte load

__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// A block's scale, from the bits of its largest magnitude: NaN if one element is not finite.
// hi and lo: 2^-21 above and below 1 / s.  fp32(x / s) lies between x lo and x hi (the
// reciprocal is within 2^-23 of its exact value, each product within 2^-24 of its own), so
// where both give the same code there is no need to divide: rounding is monotonic.  They
// differ for about one element in 2^17.
struct BlockScale {
  float s, hi, lo;
  bool divide;      // a subnormal scale, whose reciprocal may overflow
};
__device__ __forceinline__ BlockScale block_scale(uint32_t top) {
  BlockScale b;
  b.s = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __fdiv_rn(__uint_as_float(top), 448.0f);
  b.divide = b.s < 1.17549435e-38f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(b.s));
  b.hi = inv * (1.0f + 4.76837158e-7f);
  b.lo = inv * (1.0f - 4.76837158e-7f);
  return b;
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Two products in one instruction.
__device__ __forceinline__ float2 mul2(float a, float b, float by) {
  float2 r;
  asm("{\n\t.reg .b64 v, s;\n\t"
      "mov.b64 v, {%2, %3};\n\t"
      "mov.b64 s, {%4, %4};\n\t"
      "mul.rn.f32x2 v, v, s;\n\t"
      "mov.b64 {%0, %1}, v;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(by));
  return r;
}
// Four codes (a scale of 0 or NaN gives zeros).
__device__ __forceinline__ uint32_t codes4(const float* f, const BlockScale& b) {
  if (!(b.s > 0.0f)) return 0u;
  auto codes = [&](float by) {
    const float2 a = mul2(f[0], f[1], by), c = mul2(f[2], f[3], by);
    return e4m3x2(a.x, a.y) | (e4m3x2(c.x, c.y) << 16);
  };
  const uint32_t hi = codes(b.hi), lo = codes(b.lo);
  if (hi == lo && !b.divide) return hi;
  return e4m3x2(__fdiv_rn(f[0], b.s), __fdiv_rn(f[1], b.s)) | (e4m3x2(__fdiv_rn(f[2], b.s), __fdiv_rn(f[3], b.s)) << 16);
}
__device__ __forceinline__ uint8_t code1(float f, const BlockScale& b) {
  return b.s > 0.0f ? uint8_t(e4m3x2(__fdiv_rn(f, b.s), 0.0f)) : uint8_t(0);
}

// The codes of a vector.
template <typename T>
__device__ __forceinline__ void put_codes(uint8_t* dst, const uint4& v, const BlockScale& b) {
  float f[kVec<T>];
  Elem<T>::unpack(v, f);
  if constexpr (kVec<T> == 4) *reinterpret_cast<uint32_t*>(dst) = codes4(f, b);
  else *reinterpret_cast<uint2*>(dst) = make_uint2(codes4(f, b), codes4(f + 4, b));
}

// ------------------------------------------------------------------ quantize

constexpr int kQThreads = 256;

// Blocks of one row, eight lanes a block and sixteen elements a lane (what a block costs
// beside its elements, the scale above all, is shared by as many; four lanes were no faster).
// The vectors stay as they were loaded until their codes are made.  4096 x 4096 takes 13.9 us
// from 16-bit types (3.6 TB/s: issue slots 75 % taken while a CTA runs, 56 % of the time with start
// and end, DRAM 25 %; waits for loads are the largest stall), 14.6 from fp32 (5.8 TB/s).  VEC:
// rows start on vector boundaries; else element by element.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads) fp8_rows_kernel(const T* __restrict__ x, int rows, int cols,
                                                             uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int kLanes = 8, kMine = kFp8Block / kLanes;
  constexpr int V = VEC ? kVec<T> : 1;
  constexpr int kLoads = kMine / V;
  constexpr int kGroups = kQThreads / kLanes;
  grid_dep_wait();
  const int kb = (cols + kFp8Block - 1) / kFp8Block;
  const int64_t blocks = int64_t(rows) * kb;
  const int l = threadIdx.x % kLanes;
  const int64_t stride = int64_t(gridDim.x) * kGroups;
  // every lane of a warp takes part in the shuffles: the last round may have no block
  for (int64_t first = int64_t(blockIdx.x) * kGroups + (threadIdx.x & ~31) / kLanes; first < blocks; first += stride) {
    const int64_t b = first + (threadIdx.x & 31) / kLanes;
    const int64_t row = blocks <= 0xffffffffll ? int64_t(uint32_t(b) / uint32_t(kb)) : b / kb;
    const int c0 = int(b - row * kb) * kFp8Block;
    const int n = b < blocks ? min(kFp8Block, cols - c0) : 0;
    const int64_t at = row * cols + c0;
    uint4 v[VEC ? kLoads : 1];
    float f[VEC ? V : kMine];
    uint32_t top = 0;
    if (VEC) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int c = (i * kLanes + l) * V;
        v[i] = c < n ? __ldg(reinterpret_cast<const uint4*>(x + at + c)) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) top = Elem<T>::larger(v[i], top);
      top = Elem<T>::as_float(top);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) f[i] = i * kLanes + l < n ? Elem<T>::one(x + at + i * kLanes + l) : 0.0f;
#pragma unroll
      for (int i = 0; i < kMine; ++i) top = max(top, magnitude(f[i]));
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const BlockScale s = block_scale(top);
    if (l == 0 && n > 0) scales[b] = s.s;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * kLanes + l) * V;
      if (c >= n) continue;
      if constexpr (VEC) put_codes<T>(codes + at + c, v[i], s);
      else codes[at + c] = code1(f[i], s);
    }
  }
}

// Blocks of 128 x 128, a CTA each, kept in registers between the maximum and the codes: three
// CTAs an SM of fp32 (a third one took 11008 x 4096 from 46.5 to 38.4 us, 5.9 TB/s), four of
// 16-bit types (30 us, 4.5 TB/s).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads, VEC ? (sizeof(T) == 4 ? 3 : 4) : 2) fp8_tile_kernel(const T* __restrict__ x, int rows, int cols, int kb,
                                                             uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int V = VEC ? kVec<T> : 4;
  constexpr int kPer = kFp8Block / V;                        // vectors of a row
  constexpr int kKeep = kFp8Block * kPer / kQThreads;        // and of a thread
  grid_dep_wait();
  const int br = blockIdx.x / kb, bc = blockIdx.x - br * kb;
  const int64_t r0 = int64_t(br) * kFp8Block;
  const int c0 = bc * kFp8Block;
  const int t = threadIdx.x;
  uint4 v[VEC ? kKeep : 1];
  float f[VEC ? 1 : kKeep][V];
  uint32_t top = 0;
  if (VEC) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int at = t + i * kQThreads, c = c0 + at % kPer * V;
      const int64_t r = r0 + at / kPer;
      v[i] = r < rows && c < cols ? __ldg(reinterpret_cast<const uint4*>(x + r * cols + c)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) top = Elem<T>::larger(v[i], top);
    top = Elem<T>::as_float(top);
  } else {
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int at = t + (i * V + j) * kQThreads, c = c0 + at % kFp8Block;
        const int64_t r = r0 + at / kFp8Block;
        f[i][j] = r < rows && c < cols ? Elem<T>::one(x + r * cols + c) : 0.0f;
        top = max(top, magnitude(f[i][j]));
      }
  }
  __shared__ uint32_t part[kQThreads / 32];
  top = __reduce_max_sync(0xffffffffu, top);
  if ((t & 31) == 0) part[t >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQThreads / 32; ++i) top = max(top, part[i]);
  const BlockScale s = block_scale(top);
  if (t == 0) scales[blockIdx.x] = s.s;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    if constexpr (VEC) {
      const int at = t + i * kQThreads, c = c0 + at % kPer * V;
      const int64_t r = r0 + at / kPer;
      if (r < rows && c < cols) put_codes<T>(codes + r * cols + c, v[i], s);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int at = t + (i * V + j) * kQThreads, c = c0 + at % kFp8Block;
        const int64_t r = r0 + at / kFp8Block;
        if (r < rows && c < cols) codes[r * cols + c] = code1(f[i][j], s);
      }
    }
  }
}

void pdl_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned grid, unsigned threads, cudaStream_t st) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(grid, 1, 1);
  cfg->blockDim = dim3(threads, 1, 1);
  cfg->stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = prof_on() ? 0 : 1;
}

template <typename T>
cudaError_t quantize_t(const void* x, int64_t rows, int64_t cols, int block_rows, uint8_t* codes, float* scales, int sms,
                       cudaStream_t st) {
  const T* xt = static_cast<const T*>(x);
  const bool vec = cols % kVec<T> == 0;
  const int64_t kb = (cols + kFp8Block - 1) / kFp8Block;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  if (block_rows == 1) {
    constexpr int64_t per = kQThreads / 8;
    pdl_config(&cfg, attr, unsigned(std::min<int64_t>((rows * kb + per - 1) / per, int64_t(sms) * 32)), kQThreads, st);
    return vec ? cudaLaunchKernelEx(&cfg, fp8_rows_kernel<T, true>, xt, int(rows), int(cols), codes, scales)
               : cudaLaunchKernelEx(&cfg, fp8_rows_kernel<T, false>, xt, int(rows), int(cols), codes, scales);
  }
  const int64_t tiles = (rows + kFp8Block - 1) / kFp8Block * kb;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  pdl_config(&cfg, attr, unsigned(tiles), kQThreads, st);
  return vec ? cudaLaunchKernelEx(&cfg, fp8_tile_kernel<T, true>, xt, int(rows), int(cols), int(kb), codes, scales)
             : cudaLaunchKernelEx(&cfg, fp8_tile_kernel<T, false>, xt, int(rows), int(cols), int(kb), codes, scales);
}

// ------------------------------------------------------------------ dequantize

__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* o, float v) { *o = __float2half_rn(v); }

__device__ __forceinline__ float2 values2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(two), __NV_E4M3);
  return __half22float2(__half2(h));
}

// V codes a thread, in one row (the row length is a multiple of V): 16 bytes of results, so
// that a warp writes whole lines (16 codes a thread: 51 us against 46 for 11008 x 4096 in
// fp32, 4.9 TB/s, most of it writes; issue 56 %, a load in flight a thread).
template <typename T, int V>
__global__ void __launch_bounds__(kQThreads) fp8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                   const float* __restrict__ scales, int64_t rows, int cols,
                                                                   int row_shift, T* __restrict__ out) {
  grid_dep_wait();
  const int kb = (cols + kFp8Block - 1) / kFp8Block, per = cols / V;
  const int64_t total = rows * per;
  for (int64_t i = int64_t(blockIdx.x) * kQThreads + threadIdx.x; i < total; i += int64_t(gridDim.x) * kQThreads) {
    const int64_t row = i / per;
    const int c = int(i - row * per) * V;
    const float s = __ldg(scales + (row >> row_shift) * kb + c / kFp8Block);
    if constexpr (V > 1) {
      uint32_t w[V / 4];
      if constexpr (V == 4) w[0] = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
      else *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(codes) + i);
      alignas(16) T v[V];
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 f = values2((w[j / 2] >> (16 * (j & 1))) & 0xffffu);
        put(&v[2 * j], __fmul_rn(f.x, s));
        put(&v[2 * j + 1], __fmul_rn(f.y, s));
      }
      uint4* o = reinterpret_cast<uint4*>(out + i * V);
#pragma unroll
      for (int j = 0; j < int(sizeof(v) / 16); ++j) o[j] = reinterpret_cast<const uint4*>(v)[j];
    } else {
      put(out + i, __fmul_rn(values2(__ldg(codes + i)).x, s));
    }
  }
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols, int block_rows, void* out,
                         int sms, cudaStream_t st) {
  constexpr int V = kVec<T>;
  const bool vec = cols % V == 0;
  const int64_t work = rows * cols / (vec ? V : 1);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, unsigned(std::max<int64_t>(1, std::min<int64_t>((work + kQThreads - 1) / kQThreads, int64_t(sms) * 32))),
             kQThreads, st);
  const int shift = block_rows == 1 ? 0 : 7;
  T* o = static_cast<T*>(out);
  return vec ? cudaLaunchKernelEx(&cfg, fp8_dequantize_kernel<T, V>, codes, scales, rows, int(cols), shift, o)
             : cudaLaunchKernelEx(&cfg, fp8_dequantize_kernel<T, 1>, codes, scales, rows, int(cols), shift, o);
}

// ------------------------------------------------------------------ linear, few tokens

// y for a few tokens: the weight bytes are the whole cost.  A CTA holds the codes of all
// tokens in shared memory, quantized here unless they came so, and takes 16 weight rows at
// a time, its eight warps an eighth of the blocks along K each.  The weight goes from global
// memory into the A fragments of mma.sync m16n8k32 (e4m3): the k order inside a block is
// free as long as both operands agree, so a lane's share of a row and block is two pieces
// of 16 contiguous bytes, and the four lanes of a row load 64.  A block's sum is scaled and
// added in fp32; the warps meet in shared memory.  Bound by DRAM and its latency: 4096 x 4096
// with one token 6.2 us (2.7 TB/s), 32768 x 8192 53 us (5.1 TB/s).
constexpr int kSmWarps = 8;
constexpr int kSmThreads = 32 * kSmWarps;
constexpr int kSmAhead = 4;                        // blocks whose loads are in flight

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void store_y(const Fp8LinearArgs& a, int64_t m, int64_t n, float v) {
  const int64_t at = m * a.N + n;
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

// Shared memory: codes [M][kb * 128 + 64] (64: neighbouring tokens lie in other banks),
// scales [kb][8] (those past M are never used), partial sums [warp][8][16 rows].
__host__ __device__ constexpr size_t small_smem(int m, int kb) {
  return size_t(m) * (size_t(kb) * 128 + 64) + size_t(kb) * 8 * 4 + size_t(kSmWarps) * 16 * 8 * 4;
}

template <typename T>
__global__ void __launch_bounds__(kSmThreads) fp8_small_kernel(const Fp8LinearArgs a, const T* __restrict__ x,
                                                               const float* __restrict__ given_scale) {
  extern __shared__ __align__(16) uint8_t codes[];
  constexpr int NP = 8;
  const int K = int(a.K), M = int(a.M);
  const int kb = (K + kFp8Block - 1) / kFp8Block;
  const int stride = kb * 128 + 64;
  float* sx = reinterpret_cast<float*>(codes + size_t(M) * stride);
  float* part = sx + kb * NP;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, q = lane & 3;
  grid_dep_wait();
  const int groups = int((a.N + kFp8SmallRows - 1) / kFp8SmallRows);
  const int b0 = kb * warp / kSmWarps, b1 = kb * (warp + 1) / kSmWarps;   // this warp's blocks
  uint4 wv[kSmAhead][2][2];                        // block, row (g, g + 8), 64-byte half
  auto load_w = [&](int grp, int b) {
#pragma unroll
    for (int j = 0; j < kSmAhead; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t n = min(int64_t(grp) * 16 + 8 * h + g, a.N - 1);
        const int k = (b + j) * kFp8Block + 16 * q;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          wv[j][h][i] = b + j < b1 && k + 64 * i < K ? __ldg(reinterpret_cast<const uint4*>(a.w + n * K + k + 64 * i))
                                                    : make_uint4(0u, 0u, 0u, 0u);
      }
  };
  int grp = blockIdx.x;
  load_w(grp, b0);

  // The tokens' codes and scales; several loads of a thread in flight.  K is a multiple of 16,
  // a row's last block is filled up with zeros.
  if constexpr (sizeof(T) == 1) {
    for (int i = t; i < M * kb * 8; i += kSmThreads) {
      const int m = i / (kb * 8), v = i - m * (kb * 8);
      *reinterpret_cast<uint4*>(codes + m * stride + 16 * v) =
          16 * v < K ? __ldg(reinterpret_cast<const uint4*>(x + int64_t(m) * K) + v) : make_uint4(0u, 0u, 0u, 0u);
    }
    for (int i = t; i < M * kb; i += kSmThreads) sx[i % kb * NP + i / kb] = __ldg(given_scale + i);
  } else {
    constexpr int kBatch = 4;
    for (int i0 = warp; i0 < M * kb; i0 += kSmWarps * kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * kSmWarps, m = i / kb, k = (i - m * kb) * kFp8Block + 4 * lane;
        raw[j] = make_uint4(0u, 0u, 0u, 0u);
        if (m < M && k < K) {
          if constexpr (sizeof(T) == 4) {
            raw[j] = __ldg(reinterpret_cast<const uint4*>(x + int64_t(m) * K + k));
          } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(x + int64_t(m) * K + k));
            raw[j].x = v.x;
            raw[j].y = v.y;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * kSmWarps, m = i / kb, b = i - m * kb;
        if (m >= M) break;
        float f[kVec<T>];                          // four elements
        Elem<T>::unpack(raw[j], f);
        const uint32_t top = max(max(magnitude(f[0]), magnitude(f[1])), max(magnitude(f[2]), magnitude(f[3])));
        const BlockScale s = block_scale(__reduce_max_sync(0xffffffffu, top));
        *reinterpret_cast<uint32_t*>(codes + m * stride + b * kFp8Block + 4 * lane) = codes4(f, s);
        if (lane == 0) sx[b * NP + m] = s.s;
      }
    }
  }
  __syncthreads();

  for (; grp < groups; grp += gridDim.x) {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const float* ws = a.w_scale + int64_t(grp / 8) * kb;   // sixteen rows lie in one block of 128
    for (int b = b0; b < b1; b += kSmAhead) {
#pragma unroll
      for (int j = 0; j < kSmAhead; ++j) {
        if (b + j >= b1) break;
        const float sw = __ldg(ws + b + j);
        const uint32_t r0[8] = {wv[j][0][0].x, wv[j][0][0].y, wv[j][0][0].z, wv[j][0][0].w,
                                wv[j][0][1].x, wv[j][0][1].y, wv[j][0][1].z, wv[j][0][1].w};
        const uint32_t r1[8] = {wv[j][1][0].x, wv[j][1][0].y, wv[j][1][0].z, wv[j][1][0].w,
                                wv[j][1][1].x, wv[j][1][1].y, wv[j][1][1].z, wv[j][1][1].w};
        uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
        if (g < M) {
          const uint4* xc = reinterpret_cast<const uint4*>(codes + g * stride + (b + j) * kFp8Block + 16 * q);
          x0 = xc[0], x1 = xc[4];
        }
        const uint32_t xw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_e4m3(d, r0[2 * i], r1[2 * i], r0[2 * i + 1], r1[2 * i + 1], xw[2 * i], xw[2 * i + 1]);
        const float2 s = *reinterpret_cast<const float2*>(sx + (b + j) * NP + 2 * q);
        acc[0] = fmaf(d[0], s.x * sw, acc[0]);
        acc[1] = fmaf(d[1], s.y * sw, acc[1]);
        acc[2] = fmaf(d[2], s.x * sw, acc[2]);
        acc[3] = fmaf(d[3], s.y * sw, acc[3]);
      }
      if (b + kSmAhead < b1) load_w(grp, b + kSmAhead);
    }
    if (grp + int(gridDim.x) < groups) load_w(grp + int(gridDim.x), b0);
    float* mine = part + warp * (16 * NP);         // [token][row]
    mine[(2 * q) * 16 + g] = acc[0];
    mine[(2 * q + 1) * 16 + g] = acc[1];
    mine[(2 * q) * 16 + g + 8] = acc[2];
    mine[(2 * q + 1) * 16 + g + 8] = acc[3];
    __syncthreads();
    for (int i = t; i < 16 * M; i += kSmThreads) {
      float v = 0.0f;
#pragma unroll
      for (int wp = 0; wp < kSmWarps; ++wp) v += part[wp * (16 * NP) + i];
      const int64_t n = int64_t(grp) * 16 + (i & 15);
      if (n < a.N) store_y(a, i >> 4, n, v);
    }
    __syncthreads();   // part may be written again
  }
}

template <typename T>
cudaError_t small_t(const Fp8LinearArgs& a, const void* x, const float* scale, int sms, cudaStream_t st) {
  static PerDeviceOnce attr_done;
  const int dev = PerDeviceOnce::current();
  if (!attr_done.done(dev)) {
    const cudaError_t e = cudaFuncSetAttribute(fp8_small_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
    attr_done.mark(dev);
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, unsigned(fp8_small_ctas(a.N, sms)), kSmThreads, st);
  cfg.dynamicSmemBytes = small_smem(int(a.M), int((a.K + kFp8Block - 1) / kFp8Block));
  return cudaLaunchKernelEx(&cfg, fp8_small_kernel<T>, a, static_cast<const T*>(x), scale);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* x, int in_dtype, int64_t rows, int64_t cols, int block_rows, uint8_t* codes,
                                float* scales, int sms, cudaStream_t st, int* launches) {
  NF4_PROF_BEGIN(st, kKFp8Quantize);
  cudaError_t e = in_dtype == NF4_F32   ? quantize_t<float>(x, rows, cols, block_rows, codes, scales, sms, st)
                  : in_dtype == NF4_F16 ? quantize_t<__half>(x, rows, cols, block_rows, codes, scales, sms, st)
                                        : quantize_t<__nv_bfloat16>(x, rows, cols, block_rows, codes, scales, sms, st);
  NF4_PROF_END(st, kKFp8Quantize);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols, int block_rows,
                                  int out_dtype, void* out, int sms, cudaStream_t st, int* launches) {
  NF4_PROF_BEGIN(st, kKFp8Dequantize);
  cudaError_t e = out_dtype == NF4_F32   ? dequantize_t<float>(codes, scales, rows, cols, block_rows, out, sms, st)
                  : out_dtype == NF4_F16 ? dequantize_t<__half>(codes, scales, rows, cols, block_rows, out, sms, st)
                                         : dequantize_t<__nv_bfloat16>(codes, scales, rows, cols, block_rows, out, sms, st);
  NF4_PROF_END(st, kKFp8Dequantize);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_fp8_linear(const Fp8LinearArgs& given, const void* x, const float* x_scale, uint8_t* codes,
                              float* scales, int sms, cudaStream_t st, int* launches) {
  Fp8LinearArgs a = given;
  const bool small = fp8_streams(a.M, a.N, a.K, sms);
  const bool inside = small && x_scale == nullptr && fp8_quantizes_inside(a.M, a.N, a.K);
  a.x = x_scale != nullptr ? static_cast<const uint8_t*>(x) : codes;
  a.x_scale = x_scale != nullptr ? x_scale : scales;
  Fp8Gemm g;
  if (!small && !g.prepare(a, sms)) return cudaErrorInvalidValue;
  if (x_scale == nullptr && !inside) {
    const cudaError_t e = launch_fp8_quantize(x, a.dtype, a.M, a.K, 1, codes, scales, sms, st, launches);
    if (e != cudaSuccess) return e;
  }
  if (!small) return g.run(st, launches);
  NF4_PROF_BEGIN(st, kKFp8Linear);
  cudaError_t e = !inside              ? small_t<uint8_t>(a, a.x, a.x_scale, sms, st)
                  : a.dtype == NF4_F32 ? small_t<float>(a, x, nullptr, sms, st)
                  : a.dtype == NF4_F16 ? small_t<__half>(a, x, nullptr, sms, st)
                                       : small_t<__nv_bfloat16>(a, x, nullptr, sms, st);
  NF4_PROF_END(st, kKFp8Linear);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nf4
