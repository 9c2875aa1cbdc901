// The rank-r products of the gated feed-forward layer on the sm_100a tensor cores, both
// projections p in one launch each:
//   T_p  = s x A_p^T                 [2, M, r]
//   d_0  = dh u act'(g) (dg),  d_1 = dh act(g) (du)
//   U_p  = s d_p B_p                 [2, M, r]
//   dB_p = d_p^T T_p                 fp32 [2, N, r]
//   dA_p = U_p^T x                   fp32 [2, r, K]
// A tile is 128 rows of the result by 64 adapter columns of both projections (a further
// grid dimension for r > 64); the reduction runs in steps of 64 and is split over the CTAs
// of a cluster, which sum their fp32 partials through distributed shared memory in a fixed
// order.
//
// T and dA are fed by TMA.  U and dB make their A operand, d, on the way: sixteen warps
// read dh, g and u (copied two steps ahead), compute dg and du in fp32 and write them as
// 16-bit terms, swizzled, into shared memory (eight warps of twice the work took 118 and 117 us
// for U and dB at 4096 tokens, 11008 x 4096, against 98 and 107: a step is its arithmetic's
// latency more than its rate); U's warps store the first terms to global
// memory too, for dx.  dB computes d a second time instead of reading it: the fp32 value
// is what it needs, and dh, g and u are 3/4 of the bytes of two terms of dg and du.
//
// Measured at 4096 tokens, 11008 x 4096, r = 64: U 98 us (reads 270 MB, writes 180: 4.6 TB/s), dB
// 107 (270 MB, 2.5 TB/s), dA 25, T 16.  U and dB are bound by the latency of making d, a step's
// arithmetic and its way into shared memory (issue 32 to 38 %, DRAM 27 to 34 %), and by clusters
// that leave 20 to 52 of 148 SMs idle.
//
// Gradients are fp32, and one rounding of d or U to 16 bits would be their largest error by
// far (2^-9 against 2^-24).  So d and U enter as three bf16 terms that together hold 24
// bits, or two f16 terms, the second scaled by 2^11 (22 bits; see expert_grad.cu).  The tensor
// core truncates when it adds to an accumulator, each time by 2^-26 of it on average and
// always towards zero, so that the loss grows with the number of instructions.  So the first
// terms go by turns into two accumulators, and no more than 16 instructions into one before
// it is added to a total in fp32 (rounded) and begun anew, while the other takes the next
// ones; the small terms have a third.  At 4096 tokens, 11008 x 4096 that took dA's error from
// 2.0e-6 to 5.1e-7 and dB's from 8.2e-7 to 3.1e-7 relative to 64 bits.
#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_grad.h"
#include "gated_act.cuh"
#include "gated_rank.h"
#include "nf4_common.cuh"
#include "nf4_dequant.cuh"
#include "ring_wait.cuh"
#include "tc_common.cuh"
#include "tensor_maps.h"

namespace nf4 {
namespace {

using namespace tc;
using expert::elect_one;
using expert::pack2;
using expert::ring_wait;
using expert::unpack2;
using expert::warp_wait;

constexpr int kCols = 64;                          // adapter columns of a tile, per projection
constexpr uint32_t kTileBytes = 128 * 128;         // 128 x 64 or 64 x 128 16-bit values
constexpr uint32_t kBoxBytes = 64 * 128;           // 64 x 64
constexpr int kMaxSlices = 16;
constexpr int kWindow = 4;                         // steps (of four instructions) into an accumulator
constexpr uint32_t kParkBytes = 128 * 2 * kCols * 4;   // a CTA's partial

// The term that comes after `first` in a split of v: what rounding left.  Nothing is left
// of an infinity (whose difference to itself would be NaN).
__device__ __forceinline__ float rest(float v, float first) {
  const float d = v - first;
  return fabsf(d) < __uint_as_float(0x7f800000u) ? d : 0.0f;
}

// Four consecutive columns (`col` .. of 0 .. 2 kCols) of row `row` of the result.  T is rounded to
// the compute type, which is what the forward's MMAs and a saved t take; U's first term, of as
// many as keep its bits for dA, is what dx's MMAs take.
template <GatedRankKind KIND>
__device__ __forceinline__ void store4(const GatedRankParams& p, int row, int col, int col0, float4 v) {
  const int proj = col >= kCols ? 1 : 0;
  const int j = col0 + col - proj * kCols;
  if (j >= p.r) return;
  if (KIND == kGatedT || KIND == kGatedU) {
    if (row >= p.M) return;
    const bool f16 = p.f16 != 0;
    float u[4] = {v.x * p.scale, v.y * p.scale, v.z * p.scale, v.w * p.scale};
    const int terms = KIND == kGatedU ? p.terms : 1;
    uint16_t* o = p.out16 + (int64_t(proj) * terms * p.M + row) * p.r + j;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (i >= terms) break;
      const uint2 w = make_uint2(pack2(f16, u[0], u[1]), pack2(f16, u[2], u[3]));
      *reinterpret_cast<uint2*>(o + int64_t(i) * p.M * p.r) = w;
      const float2 a = unpack2(f16, w.x), b = unpack2(f16, w.y);
      const float rounded[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = rest(u[e], rounded[e]) * (f16 ? kULoMul : 1.0f);
    }
  } else if (KIND == kGatedDB) {
    if (row < p.N) *reinterpret_cast<float4*>(p.out32 + (int64_t(proj) * p.N + row) * p.r + j) = v;
  } else {
    if (row >= p.K) return;
    float* o = p.out32 + (int64_t(proj) * p.r + j) * p.K + row;
    o[0] = v.x;
    o[int64_t(p.K)] = v.y;
    o[2 * int64_t(p.K)] = v.z;
    o[3 * int64_t(p.K)] = v.w;
  }
}

__device__ __forceinline__ void add32(uint32_t at, float (&f)[32]) {
  uint32_t v[32];
  tmem_ld_32x32b_x32(at, v);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] += __uint_as_float(v[i]);
}

// A CTA's sums of 32 columns, lane = row: the accumulators joined.  at: TMEM address of the
// first, the others `stride` further each: of even steps, odd steps and, with `make`, of the
// small terms and the total of the windows before.  `steps` of this CTA.
__device__ __forceinline__ void join_accs(uint32_t at, uint32_t stride, int steps, bool make, float lo_scale,
                                          float (&f)[32]) {
  uint32_t v[32];
  if (steps == 0) {
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = 0.0f;
    return;
  }
  tmem_ld_32x32b_x32(at, v);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
  if (steps > 1) add32(at + stride, f);
  if (make) {
    if (steps > 2 * kWindow) add32(at + 3 * stride, f);
    tmem_ld_32x32b_x32(at + 2 * stride, v);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = fmaf(__uint_as_float(v[i]), lo_scale, f[i]);
  }
}

// 32 columns at `c` of tile row `prow` to the result or, with several slices, to the parked
// partial (16-byte chunks swizzled by row).
template <GatedRankKind KIND>
__device__ __forceinline__ void finish32(const GatedRankParams& p, float* park, int row0, int prow, int c, int col0,
                                         const float (&f)[32]) {
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float4 q = make_float4(f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]);
    const int col = c + 4 * g;
    if (p.slices == 1) store4<KIND>(p, row0 + prow, col, col0, q);
    else *reinterpret_cast<float4*>(park + prow * (2 * kCols) + 4 * ((col >> 2) ^ (prow & 7))) = q;
  }
}

// The slices' partials of a tile: CTA q of the cluster sums its share of the rows over the
// slices in their order.  All threads of the CTA; the second barrier keeps the partials alive.
template <GatedRankKind KIND>
__device__ __forceinline__ void sum_slices(const GatedRankParams& p, const float* park, int row0, int col0) {
  cluster_sync();
  const int q = int(cluster_ctarank()), S = p.slices;
  const int r0 = q * 128 / S, r1 = (q + 1) * 128 / S;
  const int rows = r1 - r0;
  constexpr int kVec = 2 * kCols / 4;
  const uint32_t base = smem_u32(park);
  for (int i = threadIdx.x; i < rows * kVec; i += blockDim.x) {
    // dA: neighbouring threads on neighbouring rows, which its transposed result keeps together
    const int cv = KIND == kGatedDA ? i / rows : i % kVec;
    const int trow = r0 + (KIND == kGatedDA ? i % rows : i / kVec);
    const uint32_t off = uint32_t((trow * (2 * kCols) + 4 * (cv ^ (trow & 7))) * 4);
    float4 part[kMaxSlices], acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int sl = 0; sl < kMaxSlices; ++sl)   // all on their way before the first is needed
      if (sl < S) part[sl] = ld_shared_cluster_f4(mapa_shared(base + off, uint32_t(sl)));
#pragma unroll
    for (int sl = 0; sl < kMaxSlices; ++sl) {
      if (sl >= S) break;
      acc.x += part[sl].x;
      acc.y += part[sl].y;
      acc.z += part[sl].z;
      acc.w += part[sl].w;
    }
    store4<KIND>(p, row0 + trow, 4 * cv, col0, acc);
  }
  cluster_sync();
}

// This CTA's steps of the reduction.
struct Share {
  int step0, steps;
};
__device__ __forceinline__ Share share_of(const GatedRankParams& p) {
  const int q = blockIdx.y;
  const int s0 = int(int64_t(p.red_steps) * q / p.slices), s1 = int(int64_t(p.red_steps) * (q + 1) / p.slices);
  return Share{s0, s1 - s0};
}

// ------------------------------------------------------------------ T and dA: operands by TMA

constexpr int kTmaThreads = 256;    // A loads, B loads, MMA, TMEM; four epilogue warps
constexpr int tma_boxes(GatedRankKind kind, int terms) { return kind == kGatedT ? 2 : 2 * terms; }
constexpr uint32_t tma_stage_bytes(GatedRankKind kind, int terms) {
  return kTileBytes + uint32_t(tma_boxes(kind, terms)) * kBoxBytes;
}
constexpr int tma_stages(GatedRankKind kind) { return kind == kGatedT ? 4 : 3; }

struct TmaShared {
  uint64_t full[4];
  uint64_t empty[4];
  uint64_t accum;
  uint64_t accfull[2];        // dA: a window's MMAs finished
  uint64_t accempty[2];       // and its sums were read
  uint32_t tmem_base;
  uint32_t abort_flag;
};
constexpr size_t tma_smem(GatedRankKind kind) {
  return size_t(tma_stages(kind)) * tma_stage_bytes(kind, 3) + sizeof(TmaShared) + 1024;
}
static_assert(tma_smem(kGatedDA) <= 232448 && tma_stages(kGatedT) * tma_stage_bytes(kGatedT, 1) >= kParkBytes, "shared memory");

template <GatedRankKind KIND>
__global__ void __launch_bounds__(kTmaThreads, 1)
    gated_tma_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const GatedRankParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = expert::align_1024(smem_raw);
  constexpr int kStages = tma_stages(KIND);
  const int terms = KIND == kGatedT ? 1 : p.terms;
  const int boxes = tma_boxes(KIND, terms);
  const uint32_t stage_bytes = tma_stage_bytes(KIND, terms);
  TmaShared* sh = reinterpret_cast<TmaShared*>(smem + kStages * tma_stage_bytes(KIND, 3));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sh->abort_flag;
  const int row0 = blockIdx.x * 128;
  const int col0 = blockIdx.z * kCols;
  const Share w = share_of(p);
  constexpr uint32_t kAccCols = KIND == kGatedT ? 256 : 512;
  // T: even and odd steps; dA: even and odd windows and the small terms, each of 2 kCols columns
  constexpr uint32_t kAccStride = 2 * kCols;

  // A kernel launched as this one's programmatic dependent may start on the SMs this grid
  // leaves free; it waits for this grid before it reads the result.
  grid_dep_launch();
  if (threadIdx.x == 0) {
    tma_prefetch(&tm_a);
    tma_prefetch(&tm_b);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh->full[s], 2);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->accum, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->accfull[b], 1);
      mbar_init(&sh->accempty[b], 4);
    }
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 3) {
    tmem_alloc(&sh->tmem_base, kAccCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (warp < 2) {
    const bool issue = elect_one();
    int issued = 0, s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < w.steps; ++i) {
      if (!ring_wait(&sh->empty[s], ph, abort_flag, p.status)) break;
      if (issue) {
        uint8_t* a = smem + s * stage_bytes;
        uint8_t* b = a + kTileBytes;
        const int red0 = (w.step0 + i) * 64;
        if (warp == 0) {
          mbar_arrive_expect_tx(&sh->full[s], kTileBytes);
          if (KIND == kGatedT) {
            tma_load_2d(a, &tm_a, &sh->full[s], red0, row0);
          } else {
            tma_load_2d(a, &tm_a, &sh->full[s], row0, red0);
            tma_load_2d(a + kBoxBytes, &tm_a, &sh->full[s], row0 + 64, red0);
          }
        } else {
          mbar_arrive_expect_tx(&sh->full[s], uint32_t(boxes) * kBoxBytes);
          for (int z = 0; z < boxes; ++z) {
            if (KIND == kGatedT) tma_load_3d(b + z * kBoxBytes, &tm_b, &sh->full[s], red0, col0, z);
            else tma_load_3d(b + z * kBoxBytes, &tm_b, &sh->full[s], col0, red0, z);
          }
        }
      }
      __syncwarp();
      ++issued;
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
      }
    }
    if (*abort_flag) {   // unwind: wait (bounded) for the copies in flight
      for (int i = max(0, issued - kStages); i < issued; ++i) {
        uint32_t none = 0;
        ring_wait(&sh->full[i % kStages], (i / kStages) & 1, &none, nullptr);
      }
    }
  } else if (warp == 2) {
    const bool issue = elect_one();
    bool ok = true;
    int s = 0, issued = 0;
    uint32_t ph = 0;
    for (int i = 0; i < w.steps; ++i) {
      const int window = i / kWindow, begun = i % kWindow;
      ok = ring_wait(&sh->full[s], ph, abort_flag, p.status);
      if (KIND == kGatedDA && ok && begun == 0)
        ok = ring_wait(&sh->accempty[window & 1], uint32_t((window >> 1) & 1) ^ 1u, abort_flag, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t a_base = smem_u32(smem + s * stage_bytes);
      if (issue) {
        const uint32_t d = tmem + uint32_t((KIND == kGatedT ? i : window) & 1) * kAccStride;
        if (KIND == kGatedT) {   // both projections' rows of A lie one after another: N = 128
          const uint32_t idesc = idesc_f32acc(128, 2 * kCols, false, false, p.f16 != 0);
          const uint64_t adesc = smem_desc_sw128(a_base, 16, 1024), bdesc = smem_desc_sw128(a_base + kTileBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma_f16(d, adesc + kk * 2, bdesc + kk * 2, idesc, (i > 1 || kk > 0) ? 1u : 0u);
        } else {
          const uint32_t idesc = idesc_f32acc(128, kCols, true, true, p.f16 != 0);
          const uint64_t adesc = smem_desc_sw128(a_base, 8192, 1024), bdesc = smem_desc_sw128(a_base + kTileBytes, 8192, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint64_t bz = bdesc + uint32_t(z * terms) * (kBoxBytes >> 4) + kk * 128;
              const uint32_t dz = uint32_t(z * kCols);
              umma_f16(d + dz, adesc + kk * 128, bz, idesc, (begun > 0 || kk > 0) ? 1u : 0u);
              umma_f16(tmem + 2 * kAccStride + dz, adesc + kk * 128, bz + (kBoxBytes >> 4), idesc, (i > 0 || kk > 0) ? 1u : 0u);
              if (terms > 2) umma_f16(tmem + 2 * kAccStride + dz, adesc + kk * 128, bz + 2 * (kBoxBytes >> 4), idesc, 1u);
            }
          }
        }
        // nobody waits on the last step's stage
        if (i + 1 < w.steps) umma_commit(&sh->empty[s]);
        else if (KIND == kGatedT) umma_commit(&sh->accum);
        if (KIND == kGatedDA && (begun == kWindow - 1 || i + 1 == w.steps)) umma_commit(&sh->accfull[window & 1]);
      }
      __syncwarp();
      ++issued;
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
      }
    }
    if (issue && !ok) drain_issued(sh->empty, issued, kStages);
    else if (issue && w.steps == 0) mbar_arrive(&sh->accum);
  } else if (warp >= 4) {
    const int quad = warp - 4;
    const uint32_t at = tmem + (uint32_t(quad * 32) << 16);
    float* park = reinterpret_cast<float*>(smem);
    if (KIND == kGatedT) {
      const bool ok = warp_wait(&sh->accum, 0, abort_flag, p.status);
      tc_fence_after();
      for (int c = 0; c < 2 * kCols; c += 32) {
        float f[32];
        join_accs(at + c, kAccStride, ok ? w.steps : 0, false, 1.0f, f);
        finish32<KIND>(p, park, row0, quad * 32 + lane, c, col0, f);
      }
    } else {
      float f[2 * kCols / 32][32];
#pragma unroll
      for (int c = 0; c < 2 * kCols / 32; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) f[c][i] = 0.0f;
      bool ok = true;
      for (int i = 0; i * kWindow < w.steps; ++i) {
        ok = warp_wait(&sh->accfull[i & 1], uint32_t(i >> 1) & 1u, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2 * kCols / 32; ++c) add32(at + uint32_t(i & 1) * kAccStride + 32 * c, f[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->accempty[i & 1]);
      }
      const float lo_scale = p.f16 ? 1.0f / kULoMul : 1.0f;
#pragma unroll
      for (int c = 0; c < 2 * kCols / 32; ++c) {
        if (ok && w.steps > 0) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(at + 2 * kAccStride + 32 * c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) f[c][i] = fmaf(__uint_as_float(v[i]), lo_scale, f[c][i]);
        }
        finish32<KIND>(p, park, row0, quad * 32 + lane, 32 * c, col0, f[c]);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (p.slices > 1) sum_slices<KIND>(p, reinterpret_cast<float*>(smem), row0, col0);
  if (KIND == kGatedDA) grid_dep_wait();   // see GatedRank::run
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, kAccCols);
  }
}

// ------------------------------------------------------------------ U and dB: d made on the way

constexpr int kMkWarps = 16;                                    // they make d, and finish the tile
constexpr int kMkThreads = 32 * (kMkWarps + 2);                 // and B loads, MMA
constexpr int kMkPass = 4 * kMkWarps;                           // rows that a chunk of every thread covers
constexpr int kMkPer = 128 / kMkPass;                           // chunks of eight elements a thread has of a step
constexpr int kMkAhead = 2 * kMkPer;                            // and how many it copies ahead
constexpr uint32_t kMkInBytes = 32 * kMkWarps * 16;             // a chunk's dh, g or u, of all threads
constexpr int kMkBufs = 2;                                      // B of a step
constexpr uint32_t kMkOpBytes = 6 * kTileBytes;                 // terms of dg, then of du
constexpr uint32_t kMkBBytes = 2 * kBoxBytes;

struct MkShared {
  uint64_t opfull;            // a step's terms are written
  uint64_t opempty;           // the MMAs that read them finished
  uint64_t bfull[kMkBufs];    // a step's B boxes landed
  uint64_t bempty[kMkBufs];   // and were read
  uint64_t accum;
  uint32_t tmem_base;
  uint32_t abort_flag;
};
constexpr size_t kMkSmem = kMkOpBytes + size_t(kMkAhead) * 3 * kMkInBytes + kMkBufs * kMkBBytes + sizeof(MkShared) + 1024;
static_assert(kMkSmem <= 232448 && kMkOpBytes >= kParkBytes, "shared memory of one CTA");

// Two 16-bit values to fp32.
template <bool F16>
__device__ __forceinline__ gated::F2 wide2(uint32_t w) {
  if (F16) {
    const float2 f = unpack2(true, w);
    return gated::f2(f.x, f.y);
  }
  return gated::f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Eight values as 16-bit terms, each what the roundings before it left (f16's second one
// scaled).  Of a first term that is not finite nothing is left over.
template <bool F16>
__device__ __forceinline__ void split8(gated::F2 (&v)[4], uint4 (&term)[3]) {
  constexpr int kTerms = gated_terms(F16);
  float top = 0.0f;   // largest magnitude, NaN if there is one
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = gated::split2(v[e]);
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(f.x), "f"(f.y), "f"(top));
  }
  // from half a step above the type's largest value on, the first term is infinite
  const bool finite = top < (F16 ? 65520.0f : 3.3961775e38f);
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = gated::split2(v[e]);
      q[e] = pack2(F16, f.x, f.y);
      if (t + 1 < kTerms) {
        v[e] = gated::fma2(wide2<F16>(q[e]), gated::both(-1.0f), v[e]);
        if (F16) v[e] = gated::mul2(v[e], gated::both(kULoMul));
      }
    }
    if (t == 0 && !finite) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = gated::split2(v[e]);
        v[e] = gated::f2(fabsf(f.x) < __uint_as_float(0x7f800000u) ? f.x : 0.0f,
                         fabsf(f.y) < __uint_as_float(0x7f800000u) ? f.y : 0.0f);
      }
    }
    term[t] = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

// 16 bytes from global to shared memory, or zeros, asynchronously.
__device__ __forceinline__ void copy_ahead(uint32_t dst, const uint16_t* src, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <GatedRankKind KIND, bool F16, int ACT>
__global__ void __launch_bounds__(kMkThreads, 1)
    gated_make_kernel(const __grid_constant__ CUtensorMap tm_b, const GatedRankParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = expert::align_1024(smem_raw);
  constexpr int kTerms = gated_terms(F16);
  uint8_t* b_base = smem + kMkOpBytes;
  uint8_t* inputs = b_base + kMkBufs * kMkBBytes;
  MkShared* sh = reinterpret_cast<MkShared*>(inputs + kMkAhead * 3 * kMkInBytes);
  auto op_tile = [&](int proj, int term) { return smem + uint32_t(proj * 3 + term) * kTileBytes; };
  auto b_box = [&](int buf, int proj) { return b_base + buf * kMkBBytes + proj * kBoxBytes; };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sh->abort_flag;
  const int row0 = blockIdx.x * 128;
  const int col0 = blockIdx.z * kCols;
  const Share w = share_of(p);
  constexpr uint32_t kAccStride = 2 * kCols;

  grid_dep_launch();
  if (threadIdx.x == 0) {
    tma_prefetch(&tm_b);
    mbar_init(&sh->opfull, kMkWarps);
    mbar_init(&sh->opempty, 1);
    for (int b = 0; b < kMkBufs; ++b) {
      mbar_init(&sh->bfull[b], 1);
      mbar_init(&sh->bempty[b], 1);
    }
    mbar_init(&sh->accum, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == kMkWarps) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (warp < kMkWarps) {
    // ---------------- d of 128 x 64 (U) or 64 x 128 (dB) elements a step, as two halves of
    // 64 x 64: a thread takes chunks of eight elements (16-byte chunk t % 8) of two rows.  It
    // copies their dh, g and u to shared memory two steps ahead (as registers one step ahead
    // allowed half of the bytes in flight), and keeps a step's terms until the MMAs have read
    // the step before.
    const int tr = threadIdx.x >> 3, tc = threadIdx.x & 7;
    constexpr int kWide = 2 * kCols / (kMkWarps / 4);
    const int64_t mn = int64_t(p.M) * p.N;
    const int red0 = w.step0 * 64;
    // chunk c (row kMkPass c + t / 8 of both halves) in the first step; a step later it is
    // `ahead` further.  `left`: how far the reduction index may still go.
    const int64_t ahead = KIND == kGatedU ? 64 : int64_t(64) * p.N;
    int64_t at[kMkPer];
    int left[kMkPer];
#pragma unroll
    for (int c = 0; c < kMkPer; ++c) {
      const int half = c * kMkPass / 64, r = c * kMkPass % 64 + tr;
      const int m = KIND == kGatedU ? row0 + 64 * half + r : red0 + r;
      const int n = KIND == kGatedU ? red0 + 8 * tc : row0 + 64 * half + 8 * tc;
      at[c] = int64_t(m) * p.N + n;
      left[c] = KIND == kGatedU ? (m < p.M ? p.N - n : 0) : (n < p.N ? p.M - m : 0);
    }
    auto place = [&](int c, int i) { return uint32_t((kMkPer * i + c) % kMkAhead) * (3 * kMkInBytes) + uint32_t(threadIdx.x) * 16u; };
    auto copy = [&](int c, int i) {
      if (i < w.steps) {
        const bool there = 64 * i < left[c];
        const int64_t e = there ? at[c] + ahead * i : 0;
        const uint32_t dst = smem_u32(inputs) + place(c, i);
        copy_ahead(dst, p.dh + e, there);
        copy_ahead(dst + kMkInBytes, p.pre + e, there);
        copy_ahead(dst + 2 * kMkInBytes, p.pre + mn + e, there);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int j = 0; j < kMkAhead; ++j) copy(j % kMkPer, j / kMkPer);
    bool ok = true;
    const uint32_t acc_at = tmem + (uint32_t((warp & 3) * 32) << 16) + (warp >> 2) * kWide;
    for (int i = 0; i < w.steps; ++i) {
      // the accumulator that step i begins anew: its MMAs finished before the last step's
      // terms were written, and the next wait for this step's
      const bool drained = i >= 2 * kWindow && i % (2 * kWindow) < 2;
      if (drained) {
        tc_fence_after();
        for (int c = 0; c < kWide; c += 32) {
          uint32_t v[32];
          float f[32];
          const uint32_t total = acc_at + 3 * kAccStride + c;
          tmem_ld_32x32b_x32(acc_at + uint32_t(i & 1) * kAccStride + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]);
          if (i > 2 * kWindow) add32(total, f);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(f[e]);
          tmem_st_32x32b_x32(total, v);
          tmem_st_wait();
        }
        tc_fence_before();
      }
      uint4 term[kMkPer][2][3];
#pragma unroll
      for (int c = 0; c < kMkPer; ++c) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kMkAhead - 1) : "memory");
        const uint8_t* src = inputs + place(c, i);
        const uint4 vd = *reinterpret_cast<const uint4*>(src);
        const uint4 vg = *reinterpret_cast<const uint4*>(src + kMkInBytes);
        const uint4 vu = *reinterpret_cast<const uint4*>(src + 2 * kMkInBytes);
        const uint32_t wd[4] = {vd.x, vd.y, vd.z, vd.w}, wg[4] = {vg.x, vg.y, vg.z, vg.w}, wu[4] = {vu.x, vu.y, vu.z, vu.w};
        gated::F2 dg[4], du[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const gated::F2 dh = wide2<F16>(wd[e]);
          gated::F2 a, d;
          gated::act_grad2<ACT>(wide2<F16>(wg[e]), &a, &d);
          dg[e] = gated::mul2(gated::mul2(dh, wide2<F16>(wu[e])), d);
          du[e] = gated::mul2(dh, a);
        }
        split8<F16>(dg, term[c][0]);
        split8<F16>(du, term[c][1]);
        copy(c, i + 2);          // into the place just read
        // dx's MMAs take dg and du of the compute type: the first terms
        if (KIND == kGatedU && blockIdx.z == 0 && 64 * i < left[c]) {
          const int64_t e = at[c] + ahead * i;
          *reinterpret_cast<uint4*>(p.d + e) = term[c][0][0];
          *reinterpret_cast<uint4*>(p.d + mn + e) = term[c][1][0];
        }
      }
      if (ok) ok = warp_wait(&sh->opempty, uint32_t(i & 1) ^ 1u, abort_flag, p.status);
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < kMkPer; ++c) {
        const uint32_t off = uint32_t(c * kMkPass / 64) * kBoxBytes + sw128_offset(uint32_t(c * kMkPass % 64 + tr), uint32_t(tc));
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int e = 0; e < kTerms; ++e) *reinterpret_cast<uint4*>(op_tile(z, e) + off) = term[c][z][e];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->opfull);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // ---------------- the tile's sums: lanes by warp % 4, columns by warp / 4
    if (ok) ok = warp_wait(&sh->accum, 0, abort_flag, p.status);
    tc_fence_after();
    const int quad = warp & 3;
    for (int c = (warp >> 2) * kWide; c < (warp >> 2) * kWide + kWide; c += 32) {
      float f[32];
      join_accs(tmem + (uint32_t(quad * 32) << 16) + c, kAccStride, ok ? w.steps : 0, true, F16 ? 1.0f / kULoMul : 1.0f, f);
      finish32<KIND>(p, reinterpret_cast<float*>(smem), row0, quad * 32 + lane, c, col0, f);
    }
  } else if (warp == kMkWarps) {
    // ---------------- MMA
    const bool issue = elect_one();
    bool ok = true;
    int issued = 0;
    constexpr bool kAMn = KIND == kGatedDB;
    constexpr uint32_t idesc = idesc_f32acc(128, kCols, kAMn, true, F16);
    for (int i = 0; i < w.steps; ++i) {
      const int b = i & 1;
      const uint32_t ph = (i >> 1) & 1;
      ok = ring_wait(&sh->bfull[b], ph, abort_flag, p.status) && ring_wait(&sh->opfull, uint32_t(i & 1), abort_flag, p.status);
      if (!ok) break;
      tc_fence_after();
      if (issue) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint64_t bdesc = smem_desc_sw128(smem_u32(b_box(b, z)), 8192, 1024);
          const uint64_t adesc = kAMn ? smem_desc_sw128(smem_u32(op_tile(z, 0)), 8192, 1024)
                                      : smem_desc_sw128(smem_u32(op_tile(z, 0)), 16, 1024);
          constexpr uint32_t kASub = kAMn ? 128 : 2;
          const uint32_t dz = uint32_t(z * kCols);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            umma_f16(tmem + uint32_t(i & 1) * kAccStride + dz, adesc + kk * kASub, bdesc + kk * 128, idesc,
                     (i % (2 * kWindow) > 1 || kk > 0) ? 1u : 0u);
#pragma unroll
            for (int term = 1; term < kTerms; ++term)
              umma_f16(tmem + 2 * kAccStride + dz, adesc + uint32_t(term) * (kTileBytes >> 4) + kk * kASub, bdesc + kk * 128,
                       idesc, (i > 0 || kk > 0 || term > 1) ? 1u : 0u);
          }
        }
        // the last step's commit goes to accum (nobody waits on its tiles)
        umma_commit(i + 1 < w.steps ? &sh->opempty : &sh->accum);
        umma_commit(&sh->bempty[b]);
      }
      __syncwarp();
      ++issued;
    }
    if (issue && !ok) drain_issued(sh->bempty, issued, kMkBufs);
    else if (issue && w.steps == 0) mbar_arrive(&sh->accum);
  } else {
    // ---------------- B rows (U) or T rows (dB) of a step, both projections
    const bool issue = elect_one();
    int issued = 0;
    for (int i = 0; i < w.steps; ++i) {
      const int b = i & 1;
      if (!ring_wait(&sh->bempty[b], ((i >> 1) & 1) ^ 1, abort_flag, p.status)) break;
      if (issue) {
        mbar_arrive_expect_tx(&sh->bfull[b], kMkBBytes);
        for (int z = 0; z < 2; ++z) tma_load_3d(b_box(b, z), &tm_b, &sh->bfull[b], col0, (w.step0 + i) * 64, z);
      }
      __syncwarp();
      ++issued;
    }
    if (*abort_flag) {   // unwind: wait (bounded) for the copies in flight
      for (int i = max(0, issued - kMkBufs); i < issued; ++i) {
        uint32_t none = 0;
        ring_wait(&sh->bfull[i & 1], (i >> 1) & 1, &none, nullptr);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (p.slices > 1) sum_slices<KIND>(p, reinterpret_cast<float*>(smem), row0, col0);
  if (KIND == kGatedDB) grid_dep_wait();   // see GatedRank::run
  if (warp == kMkWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side

PerDeviceOnce g_attr_done;

// The kernels that make d: [dB][f16][activation].
const void* const kMake[] = {
    (const void*)gated_make_kernel<kGatedU, false, gated::kSilu>,  (const void*)gated_make_kernel<kGatedU, false, gated::kGeluTanh>,
    (const void*)gated_make_kernel<kGatedU, true, gated::kSilu>,   (const void*)gated_make_kernel<kGatedU, true, gated::kGeluTanh>,
    (const void*)gated_make_kernel<kGatedDB, false, gated::kSilu>, (const void*)gated_make_kernel<kGatedDB, false, gated::kGeluTanh>,
    (const void*)gated_make_kernel<kGatedDB, true, gated::kSilu>,  (const void*)gated_make_kernel<kGatedDB, true, gated::kGeluTanh>};

cudaError_t set_attrs() {
  const int dev = PerDeviceOnce::current();
  if (g_attr_done.done(dev)) return cudaSuccess;
  const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(gated_tma_kernel<kGatedT>, attr, int(tma_smem(kGatedT)));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gated_tma_kernel<kGatedDA>, attr, int(tma_smem(kGatedDA)));
  for (const void* k : kMake)
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, attr, int(kMkSmem));
  for (const void* k : {(const void*)gated_tma_kernel<kGatedT>, (const void*)gated_tma_kernel<kGatedDA>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (const void* k : kMake)
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) g_attr_done.mark(dev);
  return e;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Clusters of s CTAs that the device runs at once (GPCs hold whole clusters, so it is less
// than its SMs / s), asked once a device for the larger kernels' threads and shared memory; 0
// where it has none of that size (above eight they are not portable).
int clusters_at_once(int s, int sms) {
  static std::atomic<int> known[64][kMaxSlices + 1];
  const int dev = PerDeviceOnce::current();
  if (dev < 0 || dev >= 64) return s > 8 ? 0 : std::max(1, sms / s);
  int n = known[dev][s].load(std::memory_order_relaxed);   // one more than the answer
  if (n > 0) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, unsigned(s), 1);
  cfg.blockDim = dim3(kMkThreads, 1, 1);
  cfg.dynamicSmemBytes = kMkSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = unsigned(s);
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kMake[0], &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = s > 8 ? 0 : std::max(1, sms / s);
  }
  known[dev][s].store(n + 1, std::memory_order_relaxed);
  return n;
}

// CTAs of a cluster, up to eight or sixteen: as many as give the fewest rounds of steps, a
// CTA's start and end counted as four, two steps a CTA at least, fewer where that ties.
// Sixteen pay where few tiles have a long reduction (backward of 40 tokens, 11008 x 4096: 103 ->
// 83 us; of 300, 8000 x 512: 79 -> 66).
int pick_slices(int64_t tiles, int64_t steps, int sms) {
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= kMaxSlices && (s == 1 || steps / s >= 2); s += s < 8 ? 1 : 8) {
    const int at_once = clusters_at_once(s, sms);
    if (at_once == 0) continue;
    const int64_t cost = cdiv(tiles, at_once) * (cdiv(steps, s) + 4);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

}  // namespace

// in: kGatedDA the terms of U, kGatedDB T; d: kGatedU dg and du; out: the result.
bool GatedRank::prepare(const GatedArgs& a, GatedRankKind k, const void* in, void* d, void* out, int sms) {
  kind = k;
  const uint64_t M = uint64_t(a.M), N = uint64_t(a.N), K = uint64_t(a.K), r = uint64_t(a.r);
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  p = GatedRankParams{};
  p.M = int(a.M);
  p.N = int(a.N);
  p.K = int(a.K);
  p.r = a.r;
  p.f16 = a.f16;
  p.act = a.act;
  p.terms = gated_terms(a.f16 != 0);
  p.scale = a.s;
  p.dh = static_cast<const uint16_t*>(a.dh);
  p.pre = static_cast<const uint16_t*>(a.pre_in);
  p.d = static_cast<uint16_t*>(d);
  p.status = a.status;
  bool ok = true;
  int64_t rows = 0, red = 0;
  switch (k) {
    case kGatedT:
      ok = encode_map_2d(&ma, a.x, MapElem::k16, K, M, 64, 128, sw) && encode_map_stack(&mb, a.A, MapElem::k16, K, r, 2, 64, 64, sw);
      rows = a.M, red = a.K;
      break;
    case kGatedDA:
      ok = encode_map_2d(&ma, a.x, MapElem::k16, K, M, 64, 64, sw) &&
           encode_map_stack(&mb, in, MapElem::k16, r, M, uint64_t(2 * p.terms), 64, 64, sw);
      rows = a.K, red = a.M;
      break;
    case kGatedU:
      ok = encode_map_stack(&mb, a.B, MapElem::k16, r, N, 2, 64, 64, sw);
      rows = a.M, red = a.N;
      break;
    case kGatedDB:
      ok = encode_map_stack(&mb, in, MapElem::k16, r, M, 2, 64, 64, sw);
      rows = a.N, red = a.M;
      break;
  }
  if (k == kGatedT || k == kGatedU) p.out16 = static_cast<uint16_t*>(out);
  else p.out32 = static_cast<float*>(out);
  if (set_attrs() != cudaSuccess) return false;
  p.red_steps = int(cdiv(red, 64));
  const int64_t tiles = cdiv(rows, 128), groups = cdiv(a.r, kCols);
  p.slices = pick_slices(tiles * groups, p.red_steps, sms);
  grid = dim3(unsigned(tiles), unsigned(p.slices), unsigned(groups));
  return ok && tiles <= int64_t(0x7fffffff);
}

// beside: run beside the kernel before on the stream, which must have let this one start
// only when what it reads was complete.  dB and dA run so beside dx and each other; they wait
// for the kernel before at their end, so that what comes after them on the stream finds
// everything done.
cudaError_t GatedRank::run(cudaStream_t st, int* launches, bool beside) const {
  cudaError_t e = set_attrs();
  if (e != cudaSuccess) return e;
  const bool tma = kind == kGatedT || kind == kGatedDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(tma ? kTmaThreads : kMkThreads, 1, 1);
  cfg.dynamicSmemBytes = tma ? tma_smem(kind) : kMkSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = grid.y;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside && !prof_on() ? 2 : 1;
  const int ids[] = {kKGatedT, kKGatedDA, kKGatedU, kKGatedDB};
  NF4_PROF_BEGIN(st, ids[kind]);
  switch (kind) {
    case kGatedT: e = cudaLaunchKernelEx(&cfg, gated_tma_kernel<kGatedT>, ma, mb, p); break;
    case kGatedDA: e = cudaLaunchKernelEx(&cfg, gated_tma_kernel<kGatedDA>, ma, mb, p); break;
    default: {
      using Make = void (*)(CUtensorMap, GatedRankParams);
      e = cudaLaunchKernelEx(&cfg, reinterpret_cast<Make>(const_cast<void*>(kMake[(kind == kGatedDB ? 4 : 0) + (p.f16 ? 2 : 0) + p.act])), mb, p);
    }
  }
  NF4_PROF_END(st, ids[kind]);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nf4
