// Forward of the expert layer with few rows per expert (serving steps): the
// 4-bit weights of the experts that have rows are streamed once.
//
//   y[m, n] = sum_k W'_e[n, k] x[m, k] + sum_j T[m, j] B_e[n, j] (+ bias_e[n])
//
// The weight bytes are the whole cost, so every SM streams an equal share of
// them whatever the routing: the work is cut into units of 128 W rows x 256
// columns (16 KB of codes), ordered by row group, 128-row tile and column, and
// CTA c of G takes units [U c / G, U (c + 1) / G).  The tiles at a share's ends
// are split between CTAs: each writes its fp32 partial to the workspace and
// counts itself, and the last one sums the partials in the order of the CTAs
// (so the result does not depend on who came last) and finishes the tile.
// Nothing waits for another CTA.
//
// Inside a CTA a producer warp keeps a ring of code and x boxes in flight; 16
// warps take one 64-wide K block of a unit and 32 rows each: a code byte becomes
// two 16-bit levels with one lookup in a 256-entry table replicated per lane
// (conflict-free), the levels are A fragments of mma.sync m16n8k16 with x as B,
// and the block scale multiplies the block's fp32 sums.  So the base enters as
// level (rounded to the compute type) times scale, the product not rounded
// again, where the GEMM rounds level * scale: either is within half a step of
// the exact product.  Measured limit of the inner loop: the table lookups, one
// shared-memory wavefront per 64 codes.
//
// T = s x A_e^T comes from a small kernel launched just before, which this one
// overlaps (programmatic dependent launch) until it finishes its first tile.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_decode.h"
#include "grouped.cuh"
#include "kernels.h"
#include "nf4_common.cuh"
#include "ring_wait.cuh"
#include "tc_common.cuh"
#include "tensor_maps.h"

namespace nf4 {
namespace {

using namespace tc;
using expert::ring_wait;
using expert::warp_wait;

constexpr int kDcWarps = 16;                         // consumer warps
constexpr int kDcThreads = 32 * (kDcWarps + 1);
constexpr int kDcRows = 128;
constexpr int kDcBlocks = 4;                         // 64-wide K blocks per unit = phases
constexpr int kDcSets = 4;                           // 32-row sets
constexpr uint32_t kDcCodeBytes = kDcRows * 128;
constexpr uint32_t kLutBytes = 256 * 32 * 4;

constexpr int dc_stages(int np) { return np == 8 ? 8 : 6; }
constexpr uint32_t dc_stage_bytes(int np) { return kDcCodeBytes + uint32_t(np) * 512u; }

template <int NP>
struct DcShared {
  uint64_t full[dc_stages(NP)];
  uint64_t empty[dc_stages(NP)];
  uint32_t abort_flag;
  int last;                                          // this CTA finishes the tile
  float red[kDcBlocks][kDcRows * NP];                // the phases' sums of a tile
  GroupTable groups;
};
template <int NP>
constexpr size_t dc_smem() {
  return size_t(dc_stages(NP)) * dc_stage_bytes(NP) + kLutBytes + sizeof(DcShared<NP>) + 1024;
}
static_assert(dc_smem<16>() <= 232448 && dc_smem<8>() <= 232448, "shared memory of one CTA");

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

// Byte offset of lane's copy of the table entry for byte j of `word`.
__device__ __forceinline__ uint32_t lut_at(uint32_t word, int j, uint32_t lane4) {
  const uint32_t shifted = j == 0 ? (word << 7) : (word >> (8 * j - 7));
  return (shifted & 0x7f80u) | lane4;
}

struct Unit {
  int rt, nt, kc;   // row group, 128-row tile, K chunk
  int e;
};

template <int NP, bool F16>
__global__ void __launch_bounds__(kDcThreads, 1)
    expert_decode_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_x,
                         const DecodeParams p) {
  constexpr int kStages = dc_stages(NP);
  constexpr int NT8 = NP / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* lut = smem + kStages * dc_stage_bytes(NP);
  DcShared<NP>* sh = reinterpret_cast<DcShared<NP>*>(lut + kLutBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sh->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], kDcWarps);
    }
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch(&tm_codes);
    tma_prefetch(&tm_x);
  }
  if (warp == kDcWarps) {
    build_groups(&sh->groups, p.offsets, p.E, p.M, NP, blockIdx.x == 0 ? p.status : nullptr);
  } else {
    // Lookup table: byte (even element in the high nibble) -> two levels in the
    // compute type, one copy per lane.
    uint32_t my = 0;
#pragma unroll
    for (int c = 0; c < 16; ++c) my = (lane & 15) == c ? level_bits(c) : my;
    const float lv = __uint_as_float(my);
    for (int e = warp; e < 256; e += kDcWarps) {
      const float hi = __shfl_sync(0xffffffffu, lv, e >> 4);
      const float lo = __shfl_sync(0xffffffffu, lv, e & 15);
      reinterpret_cast<uint32_t*>(lut)[e * 32 + lane] = two_rounded<F16>(hi, lo);
    }
  }
  __syncthreads();

  const int64_t units = int64_t(sh->groups.tiles[p.E]) * p.n_tiles * p.k_chunks;
  const int64_t G = min(int64_t(gridDim.x), units);   // CTAs with work: at least one unit each
  const bool works = int64_t(blockIdx.x) < G;
  const int64_t u0 = works ? units * blockIdx.x / G : 0, u1 = works ? units * (blockIdx.x + 1) / G : 0;
  auto unit_at = [&](int64_t u) {
    Unit r;
    const int64_t tile = u / p.k_chunks;
    r.kc = int(u - tile * p.k_chunks);
    r.rt = int(tile / p.n_tiles);
    r.nt = int(tile - int64_t(r.rt) * p.n_tiles);
    r.e = expert_of_tile(&sh->groups, p.E, r.rt);
    return r;
  };
  auto advance = [&](Unit& r) {
    if (++r.kc < p.k_chunks) return;
    r.kc = 0;
    if (++r.nt < p.n_tiles) return;
    r.nt = 0;
    if (++r.rt < sh->groups.tiles[p.E]) r.e = expert_of_tile(&sh->groups, p.E, r.rt);
  };
  auto first_row = [&](const Unit& r) { return sh->groups.start[r.e] + (r.rt - sh->groups.tiles[r.e]) * NP; };

  if (warp == kDcWarps) {
    // ---------------- producer
    if (lane == 0 && u0 < u1) {
      Unit r = unit_at(u0);
      int s = 0, issued = 0;
      uint32_t ph = 1;
      for (int64_t u = u0; u < u1; ++u) {
        if (!ring_wait(&sh->empty[s], ph, abort_flag, p.status)) break;
        uint8_t* dst = smem + s * dc_stage_bytes(NP);
        mbar_arrive_expect_tx(&sh->full[s], dc_stage_bytes(NP));
        tma_load_3d(dst, &tm_codes, &sh->full[s], r.kc * 128, r.nt * kDcRows, r.e);
        tma_load_3d(dst + kDcCodeBytes, &tm_x, &sh->full[s], 0, first_row(r), r.kc * kDcBlocks);
        advance(r);
        ++issued;
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (*abort_flag)   // unwind: wait (bounded) for the copies in flight
        for (int j = max(0, issued - kStages); j < issued; ++j) {
          uint32_t none = 0;
          ring_wait(&sh->full[j % kStages], (j / kStages) & 1, &none, nullptr);
        }
    }
    return;
  }

  // ---------------- consumers: warp = (set of 32 rows, K block of the unit)
  const int set = warp & (kDcSets - 1);
  const int phase = warp >> 2;
  const int g = lane >> 2, q = lane & 3;
  const uint32_t lane4 = uint32_t(lane) << 2;
  const bool dq = p.dq != 0;
  const float s_g = dq ? __ldg(p.absmax_scale) : 0.0f;
  const int kb_per_row = p.K >> 6;
  // The four rows of this thread: two 16-row groups, W rows 2 g and 2 g + 1 of
  // each (MMA rows g and g + 8): a half-warp's code loads then hit different
  // bank groups.
  auto raw_scales = [&](const Unit& r, uint32_t (&raw)[4]) {
    const int ch = min(r.kc * kDcBlocks + phase, kb_per_row - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(r.nt * kDcRows + set * 32 + (i >> 1) * 16 + 2 * g + (i & 1), p.N - 1);
      const int64_t b = chunk_block(int64_t(r.e) * p.N + n, p.K, ch, p.bs_shift);
      raw[i] = dq ? uint32_t(__ldg(p.absmax_q + b)) : __float_as_uint(__ldg(p.absmax + b));
    }
  };

  int s = 0;
  uint32_t ph = 0;
  bool ok = true, waited = false;
  uint32_t raw[4] = {0, 0, 0, 0};
  Unit r{};
  if (u0 < u1) {
    r = unit_at(u0);
    raw_scales(r, raw);
  }
  int64_t u = u0;
  while (u < u1) {
    const Unit tile = r;                 // first unit of this CTA's part of the tile
    const int k0 = r.kc;
    const int k1 = int(min(int64_t(p.k_chunks), int64_t(k0) + (u1 - u)));
    float acc[2][NT8][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NT8; ++t) acc[i][t][0] = acc[i][t][1] = acc[i][t][2] = acc[i][t][3] = 0.0f;
    for (int kc = k0; kc < k1; ++kc, ++u) {
      float sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = dq ? __fmul_rn(float(raw[i]), s_g) : __uint_as_float(raw[i]);
      advance(r);
      if (u + 1 < u1) raw_scales(r, raw);
      if (ok) ok = warp_wait(&sh->full[s], ph, abort_flag, p.status);
      if (ok && kc * kDcBlocks + phase < kb_per_row) {
        const uint8_t* cb = smem + s * dc_stage_bytes(NP);
        const uint8_t* xt = cb + kDcCodeBytes + phase * (NP * 128);
        uint4 xl[NT8], xh[NT8];
#pragma unroll
        for (int t = 0; t < NT8; ++t) {
          xl[t] = *reinterpret_cast<const uint4*>(xt + sw128_offset(uint32_t(8 * t + g), uint32_t(2 * q)));
          xh[t] = *reinterpret_cast<const uint4*>(xt + sw128_offset(uint32_t(8 * t + g), uint32_t(2 * q + 1)));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t row = uint32_t(set * 32 + i * 16 + 2 * g);
          const uint32_t chunk = 2u * uint32_t(phase) + uint32_t(q >> 1);
          const uint2 w0 = *reinterpret_cast<const uint2*>(cb + row * 128u + ((chunk ^ (row & 7u)) << 4) + ((q & 1) << 3));
          const uint2 w1 = *reinterpret_cast<const uint2*>(cb + (row + 1) * 128u + ((chunk ^ ((row + 1) & 7u)) << 4) + ((q & 1) << 3));
          uint32_t a[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t wa = k < 2 ? w0.x : w0.y, wb = k < 2 ? w1.x : w1.y;
            const int j = (2 * k) & 3;
            a[k][0] = *reinterpret_cast<const uint32_t*>(lut + lut_at(wa, j, lane4));
            a[k][1] = *reinterpret_cast<const uint32_t*>(lut + lut_at(wb, j, lane4));
            a[k][2] = *reinterpret_cast<const uint32_t*>(lut + lut_at(wa, j + 1, lane4));
            a[k][3] = *reinterpret_cast<const uint32_t*>(lut + lut_at(wb, j + 1, lane4));
          }
#pragma unroll
          for (int t = 0; t < NT8; ++t) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_16816<F16>(d, a[0], xl[t].x, xl[t].y);
            mma_16816<F16>(d, a[1], xl[t].z, xl[t].w);
            mma_16816<F16>(d, a[2], xh[t].x, xh[t].y);
            mma_16816<F16>(d, a[3], xh[t].z, xh[t].w);
            acc[i][t][0] = fmaf(sc[2 * i], d[0], acc[i][t][0]);
            acc[i][t][1] = fmaf(sc[2 * i], d[1], acc[i][t][1]);
            acc[i][t][2] = fmaf(sc[2 * i + 1], d[2], acc[i][t][2]);
            acc[i][t][3] = fmaf(sc[2 * i + 1], d[3], acc[i][t][3]);
          }
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&sh->empty[s]);
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
      }
    }

    // ---------------- this CTA's part of the tile: the four phases meet in
    // shared memory, [token][row] so that neighbouring threads take neighbouring rows
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = set * 32 + i * 16 + 2 * g;
#pragma unroll
      for (int t = 0; t < NT8; ++t) {
        float* o = sh->red[phase] + (8 * t + 2 * q) * kDcRows + row;
        *reinterpret_cast<float2*>(o) = make_float2(acc[i][t][0], acc[i][t][2]);
        *reinterpret_cast<float2*>(o + kDcRows) = make_float2(acc[i][t][1], acc[i][t][3]);
      }
    }
    if (!waited) grid_dep_wait();   // T, and the counters' zeros, of the kernel before
    waited = true;
    named_barrier(1, 32 * kDcWarps);
    const int row0 = first_row(tile);
    const int rows = min(NP, sh->groups.start[tile.e + 1] - row0);
    const int trow = threadIdx.x & (kDcRows - 1);
    const int n = tile.nt * kDcRows + trow;
    const int tok0 = threadIdx.x >> 7;
    float v[NP / 4];
#pragma unroll
    for (int i = 0; i < NP / 4; ++i) {
      const int at = (tok0 + 4 * i) * kDcRows + trow;
      v[i] = (sh->red[0][at] + sh->red[1][at]) + (sh->red[2][at] + sh->red[3][at]);
    }
    bool finish = true;
    if (k1 - k0 < p.k_chunks) {
      // split tile: contributors are consecutive CTAs, the first from chunk 0
      const int64_t t0 = (int64_t(tile.rt) * p.n_tiles + tile.nt) * p.k_chunks, t1 = t0 + p.k_chunks;
      const int c0 = int(((t0 + 1) * G - 1) / units), c1 = int((t1 * G - 1) / units);
      float* mine = p.partials + (size_t(blockIdx.x) * 2 + (k0 == 0 ? 1 : 0)) * (kDcRows * NP);
#pragma unroll
      for (int i = 0; i < NP / 4; ++i) __stcg(mine + (tok0 + 4 * i) * kDcRows + trow, v[i]);
      __threadfence();
      named_barrier(1, 32 * kDcWarps);
      if (threadIdx.x == 0) sh->last = atomicAdd(p.counters + c0, 1) == c1 - c0;
      named_barrier(1, 32 * kDcWarps);
      finish = sh->last != 0;
      if (finish) {
        __threadfence();
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) v[i] = 0.0f;
        for (int c = c0; c <= c1; ++c) {
          const float* from = p.partials + (size_t(c) * 2 + (c == c0 ? 1 : 0)) * (kDcRows * NP);
#pragma unroll
          for (int i = 0; i < NP / 4; ++i) v[i] += __ldcg(from + (tok0 + 4 * i) * kDcRows + trow);
        }
      }
    }
    if (finish && ok && n < p.N) {
      const uint16_t* b = p.B + (int64_t(tile.e) * p.N + n) * p.r;
      float ad[NP / 4];
#pragma unroll
      for (int i = 0; i < NP / 4; ++i) ad[i] = 0.0f;
      for (int j = 0; j < p.r; j += 8) {
        const uint4 bv = __ldg(reinterpret_cast<const uint4*>(b + j));
#pragma unroll
        for (int i = 0; i < NP / 4; ++i)
          if (tok0 + 4 * i < rows)
            ad[i] = dot8<F16>(bv, __ldcg(reinterpret_cast<const uint4*>(p.T + int64_t(row0 + tok0 + 4 * i) * p.r + j)), ad[i]);
      }
      const float bias = p.bias != nullptr ? one_float<F16>(p.bias[int64_t(tile.e) * p.N + n]) : 0.0f;
#pragma unroll
      for (int i = 0; i < NP / 4; ++i)
        if (tok0 + 4 * i < rows)
          p.y[int64_t(row0 + tok0 + 4 * i) * p.N + n] = one_rounded<F16>(v[i] + ad[i] + bias);
    }
    named_barrier(1, 32 * kDcWarps);   // red and last may be written again
  }
  if (!waited) grid_dep_wait();
}

// T = s x A_e^T for a few rows: one CTA per adapter row and token, fp32 sums in
// a fixed order.  Also clears the decode kernel's counters.
constexpr int kTsThreads = 256;
template <bool F16>
__global__ void __launch_bounds__(kTsThreads)
    expert_t_small_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ A, const int32_t* __restrict__ offsets,
                          int E, int M, int K, int r, float scale, uint16_t* __restrict__ T, int* counters, int n_counters) {
  __shared__ GroupTable groups;
  __shared__ float part[kTsThreads / 32];
  grid_dep_launch();
  const int j = blockIdx.x, m = blockIdx.y;
  if (j == 0 && m == 0)
    for (int i = threadIdx.x; i < n_counters; i += kTsThreads) counters[i] = 0;
  if (threadIdx.x < 32) build_groups(&groups, offsets, E, M, 1, nullptr);
  __syncthreads();
  if (m < groups.start[0] || m >= groups.start[E]) return;
  const int e = expert_of_tile(&groups, E, m - groups.start[0]);   // tiles of one row
  const uint4* a = reinterpret_cast<const uint4*>(A + (int64_t(e) * r + j) * K);
  const uint4* xr = reinterpret_cast<const uint4*>(x + int64_t(m) * K);
  float acc = 0.0f;
#pragma unroll 4
  for (int k = threadIdx.x; k < K / 8; k += kTsThreads) acc = dot8<F16>(__ldg(a + k), __ldg(xr + k), acc);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kTsThreads / 32; ++w) v += part[w];
    T[int64_t(m) * r + j] = one_rounded<F16>(scale * v);
  }
}

PerDeviceOnce g_attr_done;

cudaError_t set_attrs() {
  const int dev = PerDeviceOnce::current();
  if (g_attr_done.done(dev)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(expert_decode_kernel<8, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(dc_smem<8>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(expert_decode_kernel<8, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(dc_smem<8>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(expert_decode_kernel<16, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(dc_smem<16>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(expert_decode_kernel<16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(dc_smem<16>()));
  if (e == cudaSuccess) g_attr_done.mark(dev);
  return e;
}

template <int NP, bool F16>
cudaError_t launch(const ExpertDecode& L, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L.grid, 1, 1);
  cfg.blockDim = dim3(kDcThreads, 1, 1);
  cfg.dynamicSmemBytes = dc_smem<NP>();
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = prof_on() ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, expert_decode_kernel<NP, F16>, L.codes, L.x, L.p);
}

}  // namespace

size_t decode_scratch_bytes() { return size_t(kDecodeMaxCtas) * (2 * kDcRows * 16 * sizeof(float) + 16); }

bool ExpertDecode::prepare(const GroupedArgs& g, const void* T, uint8_t* scratch, int sms) {
  const LinearArgs& a = g.lin;
  np = a.M <= 8 ? 8 : 16;
  f16 = a.f16 != 0;
  const uint64_t K = uint64_t(a.K), N = uint64_t(a.N), M = uint64_t(a.M), kb = K / 64;
  bool ok = encode_map_stack(&codes, a.w->codes, MapElem::kU8, K / 2, N, uint64_t(g.E), 128, kDcRows,
                             CU_TENSOR_MAP_SWIZZLE_128B);
  {  // x as [K blocks][rows][64]
    const uint64_t dims[3] = {64, M, kb}, strides[2] = {K * 2, 128};
    const uint32_t box[3] = {64, uint32_t(np), uint32_t(kDcBlocks)};
    ok = ok && encode_map(&x, a.x, MapElem::k16, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  p = DecodeParams{};
  p.M = int(a.M);
  p.E = g.E;
  p.N = int(a.N);
  p.K = int(a.K);
  p.r = a.r;
  p.n_tiles = int((a.N + kDcRows - 1) / kDcRows);
  p.k_chunks = int((a.K + 255) / 256);
  p.bs_shift = log2_block(a.w->block_size);
  p.dq = a.w->double_quant;
  p.offsets = g.offsets;
  p.absmax_q = a.w->absmax_q;
  p.absmax = a.w->absmax;
  p.absmax_scale = a.w->absmax_scale;
  p.B = static_cast<const uint16_t*>(a.B);
  p.T = static_cast<const uint16_t*>(T);
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.y = static_cast<uint16_t*>(a.y);
  p.partials = reinterpret_cast<float*>(scratch);
  p.counters = reinterpret_cast<int*>(scratch + size_t(kDecodeMaxCtas) * 2 * kDcRows * 16 * sizeof(float));
  p.status = a.status;
  const int64_t most = max_row_tiles(a.M, g.E, np) * p.n_tiles * p.k_chunks;
  grid = unsigned(std::min<int64_t>(std::min(sms, kDecodeMaxCtas), most));
  return ok;
}

cudaError_t ExpertDecode::run(cudaStream_t st, int* launches) const {
  cudaError_t e = set_attrs();
  if (e != cudaSuccess) return e;
  NF4_PROF_BEGIN(st, kKGroupedFwd);
  if (np == 8) e = f16 ? launch<8, true>(*this, st) : launch<8, false>(*this, st);
  else e = f16 ? launch<16, true>(*this, st) : launch<16, false>(*this, st);
  NF4_PROF_END(st, kKGroupedFwd);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_expert_t_small(const GroupedArgs& g, void* T, int* counters, cudaStream_t st, int* launches) {
  const LinearArgs& a = g.lin;
  const dim3 grid(unsigned(a.r), unsigned(a.M), 1);
  const auto* x = static_cast<const uint16_t*>(a.x);
  const auto* A = static_cast<const uint16_t*>(a.A);
  auto* t = static_cast<uint16_t*>(T);
  NF4_PROF_BEGIN(st, kKGroupedT);
  if (a.f16)
    expert_t_small_kernel<true><<<grid, kTsThreads, 0, st>>>(x, A, g.offsets, g.E, int(a.M), int(a.K), a.r, a.s, t, counters, kDecodeMaxCtas);
  else
    expert_t_small_kernel<false><<<grid, kTsThreads, 0, st>>>(x, A, g.offsets, g.E, int(a.M), int(a.K), a.r, a.s, t, counters, kDecodeMaxCtas);
  NF4_PROF_END(st, kKGroupedT);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nf4
