// The rank-r products of the expert layer on the sm_100a tensor cores.
//   rows       T = s x A_e^T,  U = s dy B_e           out[m, j], m a row of the batch
//   gradients  dB_e = dy^T T,  dA_e = U^T x           out[i, j] per expert, summed over its rows
// One tile is 128 rows (tokens, or the gradient's outputs) by r columns; the
// reduction runs in steps of 64 through a TMA ring and may be split over the
// CTAs of a cluster, which sum their fp32 partials through distributed shared
// memory in a fixed order.
//
// The gradients' reduction is an expert's ragged row range.  TMA boxes start at
// any row, so only the last step holds rows of the next expert: three warps
// clear them in shared memory, in both operands (a cleared row times NaN would
// still be NaN), before that step's MMAs.
//
// dA sums products of U, whose rounding to 16 bits would be the gradient's
// largest error by far (2^-8 against 2^-23 for the sums): U is kept as two
// 16-bit terms, the rounded value and 2^8 (bf16) or 2^11 (f16) times what the
// rounding left, and dA takes both in two accumulators.  They cost r more
// columns in a product that reads x once either way.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_rank.h"
#include "grouped.cuh"
#include "kernels.h"
#include "nf4_common.cuh"
#include "nf4_dequant.cuh"
#include "ring_wait.cuh"
#include "tc_common.cuh"
#include "tensor_maps.h"

namespace nf4 {
namespace {

using namespace tc;
using expert::pack2;
using expert::ring_wait;
using expert::unpack2;

constexpr int kRkThreads = 192;    // A producer, MMA, B producer / epilogue, 3 more epilogue warps
constexpr int kRkMaxStages = 4;
constexpr uint32_t kRkABytes = 128 * 128;

struct RankShared {
  uint64_t full[kRkMaxStages];
  uint64_t empty[kRkMaxStages];
  uint64_t tail;               // the last step has landed and has rows past the group
  uint64_t fixed;              // they are cleared
  uint64_t accum;
  uint32_t tmem_base;
  uint32_t abort_flag;
  GroupTable groups;
};

__host__ __device__ inline uint32_t rank_stage_bytes(int np, bool two) {
  return kRkABytes + uint32_t(np) * 128u * (two ? 2u : 1u);
}

// Four consecutive output columns of one row.
__device__ __forceinline__ void rank_store4(const RankParams& p, int64_t base, int row, int col, float4 v) {
  if (p.kind == kRankT || p.kind == kRankU) {
    const bool f16 = p.f16 != 0;
    const float4 u = make_float4(v.x * p.scale, v.y * p.scale, v.z * p.scale, v.w * p.scale);
    const uint2 hi = make_uint2(pack2(f16, u.x, u.y), pack2(f16, u.z, u.w));
    const int64_t at = int64_t(row) * p.r + col;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = hi;
    if (p.kind == kRankU) {
      const float2 a = unpack2(f16, hi.x), b = unpack2(f16, hi.y);
      const uint2 lo = make_uint2(pack2(f16, (u.x - a.x) * p.lo_mul, (u.y - a.y) * p.lo_mul),
                                  pack2(f16, (u.z - b.x) * p.lo_mul, (u.w - b.y) * p.lo_mul));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out_lo) + at) = lo;
    }
  } else if (p.kind == kRankDB) {   // [N, r] of the expert
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + base + int64_t(row) * p.r + col) = v;
  } else {                          // dA: [r, K] of the expert
    float* o = static_cast<float*>(p.out) + base + int64_t(col) * p.Mo + row;
    o[0] = v.x;
    o[int64_t(p.Mo)] = v.y;
    o[2 * int64_t(p.Mo)] = v.z;
    o[3 * int64_t(p.Mo)] = v.w;
  }
}

__global__ void __launch_bounds__(kRkThreads, 1)
    expert_rank_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                       const __grid_constant__ CUtensorMap tm_b2, const RankParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const bool grad = p.kind == kRankDB || p.kind == kRankDA;
  const bool two = p.kind == kRankDA;
  const uint32_t b_bytes = uint32_t(p.NP) * 128u;
  const uint32_t stage_bytes = rank_stage_bytes(p.NP, two);
  RankShared* sh = reinterpret_cast<RankShared*>(smem + p.stages * stage_bytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sh->abort_flag;
  const bool b_mn = p.kind != kRankT;

  // A kernel launched as this one's programmatic dependent may start on the SMs
  // this grid leaves free; it waits for this grid before it reads the result.
  grid_dep_launch();
  if (p.zero != nullptr && blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < p.zero_n; i += kRkThreads) p.zero[i] = 0;
  if (warp == 0) build_groups(&sh->groups, p.offsets, p.E, p.M, 128, blockIdx.x == 0 && blockIdx.y == 0 ? p.status : nullptr);
  __syncthreads();
  int e, row0, row_end;          // output rows of this tile (absolute tokens, or of the expert)
  if (grad) {
    e = blockIdx.x / p.row_tiles;
    row0 = (blockIdx.x % p.row_tiles) * 128;
    row_end = p.Mo;
  } else {
    if (int(blockIdx.x) >= sh->groups.tiles[p.E]) return;   // the whole cluster
    e = expert_of_tile(&sh->groups, p.E, blockIdx.x);
    row0 = sh->groups.start[e] + (blockIdx.x - sh->groups.tiles[e]) * 128;
    row_end = sh->groups.start[e + 1];
  }
  const int tok0 = sh->groups.start[e], tok1 = sh->groups.start[e + 1];
  const int red_steps = grad ? (tok1 - tok0 + 63) / 64 : p.red_steps;
  const int per = (red_steps + p.slices - 1) / p.slices;
  const int step0 = min(int(blockIdx.y) * per, red_steps);
  const int nsteps = min(step0 + per, red_steps) - step0;
  // rows of the last step that the expert holds; 64: nothing to clear
  const int tail = grad && nsteps > 0 && step0 + nsteps == red_steps ? tok1 - tok0 - (red_steps - 1) * 64 : 64;
  const int64_t out_base = grad ? int64_t(e) * p.Mo * p.r : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&sh->full[s], 2);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->tail, 1);
    mbar_init(&sh->fixed, 3);
    mbar_init(&sh->accum, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, uint32_t(p.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  const bool a_issuer = warp == 0 && lane == 0;
  const bool b_issuer = warp == 2 && lane == 0;
  if (a_issuer || b_issuer) {
    grid_dep_wait();   // gradients: T and U of the kernels before
    int issued = 0;
    for (int i = 0; i < nsteps; ++i) {
      const int s = i % p.stages;
      if (!ring_wait(&sh->empty[s], ((i / p.stages) & 1) ^ 1, abort_flag, p.status)) break;
      uint8_t* a = smem + s * stage_bytes;
      uint8_t* b = a + kRkABytes;
      const int red0 = (step0 + i) * 64;
      if (a_issuer) {
        mbar_arrive_expect_tx(&sh->full[s], kRkABytes);
        if (grad) {
          tma_load_2d(a, &tm_a, &sh->full[s], row0, tok0 + red0);
          tma_load_2d(a + 8192, &tm_a, &sh->full[s], row0 + 64, tok0 + red0);
        } else {
          tma_load_2d(a, &tm_a, &sh->full[s], red0, row0);
        }
      } else {
        mbar_arrive_expect_tx(&sh->full[s], b_bytes * (two ? 2u : 1u));
        if (p.kind == kRankT) {
          tma_load_3d(b, &tm_b, &sh->full[s], red0, 0, e);
        } else if (p.kind == kRankU) {
          for (int g = 0; g < p.NP / 64; ++g) tma_load_3d(b + g * 8192, &tm_b, &sh->full[s], 64 * g, red0, e);
        } else {
          for (int g = 0; g < p.NP / 64; ++g) {
            tma_load_2d(b + g * 8192, &tm_b, &sh->full[s], 64 * g, tok0 + red0);
            if (two) tma_load_2d(b + b_bytes + g * 8192, &tm_b2, &sh->full[s], 64 * g, tok0 + red0);
          }
        }
      }
      ++issued;
    }
    if (*abort_flag) {   // unwind: wait (bounded) for this issuer's copies in flight
      for (int i = issued - 1; i >= 0 && i >= issued - p.stages; --i) {
        uint32_t none = 0;
        ring_wait(&sh->full[i % p.stages], (i / p.stages) & 1, &none, nullptr);
      }
    }
  }
  if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f32acc(128, p.NP, grad, b_mn, p.f16 != 0);
      bool ok = true;
      int issued = 0;
      for (int i = 0; i < nsteps; ++i) {
        const int s = i % p.stages;
        ok = ring_wait(&sh->full[s], (i / p.stages) & 1, abort_flag, p.status);
        if (ok && tail < 64 && i == nsteps - 1) {
          mbar_arrive(&sh->tail);
          ok = ring_wait(&sh->fixed, 0, abort_flag, p.status);
        }
        if (!ok) break;
        tc_fence_after();
        const uint32_t a_base = smem_u32(smem + s * stage_bytes);
        const uint32_t b_base = a_base + kRkABytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t adesc = grad ? smem_desc_sw128(a_base + kk * 2048, 8192, 1024)
                                      : smem_desc_sw128(a_base + kk * 32, 16, 1024);
          const uint64_t bdesc = b_mn ? smem_desc_sw128(b_base + kk * 2048, 8192, 1024)
                                      : smem_desc_sw128(b_base + kk * 32, 16, 1024);
          const uint32_t acc = (i > 0 || kk > 0) ? 1u : 0u;
          umma_f16(tmem, adesc, bdesc, idesc, acc);
          if (two) umma_f16(tmem + p.NP, adesc, smem_desc_sw128(b_base + b_bytes + kk * 2048, 8192, 1024), idesc, acc);
        }
        // the last step's commit goes to accum (nobody waits on its stage)
        umma_commit(i + 1 < nsteps ? &sh->empty[s] : &sh->accum);
        ++issued;
      }
      if (!ok) drain_issued(sh->empty, issued, p.stages);
      else if (nsteps == 0) mbar_arrive(&sh->accum);
    }
  } else if (warp >= 2) {
    // The last step's rows of another expert: cleared once they have landed (the
    // MMA thread, which follows the ring, says so).
    if (warp >= 3 && tail < 64) {
      const bool ok = __all_sync(0xffffffffu, ring_wait(&sh->tail, 0, abort_flag, p.status));
      if (ok) {
        uint8_t* a = smem + ((nsteps - 1) % p.stages) * stage_bytes;
        const int blocks = 2 + (p.NP / 64) * (two ? 2 : 1);   // [64 rows][128 bytes] each, A then B
        const int chunks = (64 - tail) * 8;
        for (int b = 0; b < blocks; ++b)
          for (int c = (warp - 3) * 32 + lane; c < chunks; c += 96)
            *reinterpret_cast<uint4*>(a + b * 8192 + tail * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&sh->fixed);
    }
    // epilogue warps 2..5 -> TMEM lane quadrants 2, 3, 0, 1
    const bool ok = __all_sync(0xffffffffu, ring_wait(&sh->accum, 0, abort_flag, p.status));
    tc_fence_after();
    const int quad = warp & 3;
    const int prow = quad * 32 + lane;
    const int row = row0 + prow;
    float* dst = reinterpret_cast<float*>(smem) + prow * p.NP;   // parked partial, chunks swizzled by row
    for (int c = 0; c < p.NP / 32; ++c) {
      if (p.slices == 1 && c * 32 >= p.r) break;
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + c * 32, v);
      tmem_ld_wait();
      if (two) {
        uint32_t w[32];
        tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + p.NP + c * 32, w);
        tmem_ld_wait();
#pragma unroll
        for (int u = 0; u < 32; ++u)
          v[u] = __float_as_uint(fmaf(__uint_as_float(w[u]), p.lo_scale, __uint_as_float(v[u])));
      }
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ok && nsteps > 0)
          f = make_float4(__uint_as_float(v[4 * g]), __uint_as_float(v[4 * g + 1]), __uint_as_float(v[4 * g + 2]),
                          __uint_as_float(v[4 * g + 3]));
        const int col = c * 32 + 4 * g;
        if (p.slices == 1) {
          if (col < p.r && row < row_end) rank_store4(p, out_base, row, col, f);
        } else {
          *reinterpret_cast<float4*>(dst + 4 * ((col >> 2) ^ (prow & 7))) = f;
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (p.slices > 1) {
    // CTA q of the cluster sums rows [q 128 / S, (q + 1) 128 / S) over the
    // slices in their order; the second barrier keeps the partials alive.
    cluster_sync();
    const uint32_t q = cluster_ctarank();
    const int rows_per = 128 / p.slices;
    const int vec = p.r / 4;
    const uint32_t base = smem_u32(smem);
    for (int i = threadIdx.x; i < rows_per * vec; i += blockDim.x) {
      const int cv = p.kind == kRankDA ? i / rows_per : i % vec;   // dA: consecutive threads on consecutive rows
      const int rr = p.kind == kRankDA ? i % rows_per : i / vec;
      const int trow = int(q) * rows_per + rr;
      const uint32_t off = uint32_t((trow * p.NP + 4 * (cv ^ (trow & 7))) * 4);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int sl = 0; sl < p.slices; ++sl) {
        const float4 v = ld_shared_cluster_f4(mapa_shared(base + off, uint32_t(sl)));
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      if (row0 + trow < row_end) rank_store4(p, out_base, row0 + trow, 4 * cv, acc);
    }
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, uint32_t(p.tmem_cols));
  }
}

PerDeviceOnce g_attr_done;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

bool ExpertRank::prepare(const GroupedArgs& g, RankKind kind, const void* in16, const void* in16_lo, void* out,
                         void* out_lo) {
  const LinearArgs& a = g.lin;
  const bool grad = kind == kRankDB || kind == kRankDA;
  const bool two = kind == kRankDA;
  const uint64_t M = uint64_t(a.M), N = uint64_t(a.N), K = uint64_t(a.K), E = uint64_t(g.E), r = uint64_t(a.r);
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  p = RankParams{};
  p.kind = kind;
  p.r = a.r;
  p.NP = int(cdiv(a.r, 64) * 64);
  p.E = g.E;
  p.M = int(a.M);
  p.f16 = a.f16;
  p.scale = a.s;
  p.lo_mul = a.f16 ? 2048.0f : 256.0f;
  p.lo_scale = 1.0f / p.lo_mul;
  p.offsets = g.offsets;
  p.out = out;
  p.out_lo = out_lo;
  p.status = a.status;
  bool ok = true;
  switch (kind) {
    case kRankT:
      ok = encode_map_2d(&ma, a.x, MapElem::k16, K, M, 64, 128, sw) &&
           encode_map_stack(&mb, a.A, MapElem::k16, K, r, E, 64, uint32_t(p.NP), sw);
      p.red_steps = int(cdiv(a.K, 64));
      break;
    case kRankU:
      ok = encode_map_2d(&ma, a.dy, MapElem::k16, N, M, 64, 128, sw) &&
           encode_map_stack(&mb, a.B, MapElem::k16, r, N, E, 64, 64, sw);
      p.red_steps = int(cdiv(a.N, 64));
      break;
    case kRankDB:
      ok = encode_map_2d(&ma, a.dy, MapElem::k16, N, M, 64, 64, sw) &&
           encode_map_2d(&mb, in16, MapElem::k16, r, M, 64, 64, sw);
      p.Mo = int(a.N);
      break;
    case kRankDA:
      ok = encode_map_2d(&ma, a.x, MapElem::k16, K, M, 64, 64, sw) &&
           encode_map_2d(&mb, in16, MapElem::k16, r, M, 64, 64, sw);
      p.Mo = int(a.K);
      break;
  }
  mb2 = mb;
  if (two) ok = ok && encode_map_2d(&mb2, in16_lo, MapElem::k16, r, M, 64, 64, sw);
  if (!ok) return false;
  int64_t tiles, steps;
  if (grad) {
    p.row_tiles = int(cdiv(p.Mo, 128));
    tiles = int64_t(p.row_tiles) * g.E;
    steps = cdiv(a.M, 64 * int64_t(g.E));   // of an average expert
  } else {
    tiles = max_row_tiles(a.M, g.E, 128);
    steps = p.red_steps;
  }
  if (tiles > int64_t(0x7fffffff)) return false;
  // one wave of about two CTAs per SM of a 148-SM part, four steps a slice at least
  const int64_t cap = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(296 / std::max<int64_t>(tiles, 1), 8), steps / 4));
  p.slices = 1;
  while (p.slices * 2 <= cap) p.slices *= 2;
  const uint32_t stage = rank_stage_bytes(p.NP, two);
  p.stages = int(std::min<uint32_t>(kRkMaxStages, 200u * 1024u / stage));
  p.tmem_cols = 64;
  while (p.tmem_cols < p.NP * (two ? 2 : 1)) p.tmem_cols *= 2;
  smem = size_t(p.stages) * stage + sizeof(RankShared) + 1024;
  grid = dim3(unsigned(tiles), unsigned(p.slices), 1);
  return true;
}

cudaError_t ExpertRank::run(cudaStream_t st, int* launches, bool pdl) const {
  const int dev = PerDeviceOnce::current();
  cudaError_t e = cudaSuccess;
  if (!g_attr_done.done(dev)) {
    e = cudaFuncSetAttribute(expert_rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e != cudaSuccess) return e;
    g_attr_done.mark(dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRkThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = grid.y;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl && !prof_on() ? 2 : 1;
  static const int ids[4] = {kKGroupedT, kKGroupedU, kKGroupedDB, kKGroupedDA};
  NF4_PROF_BEGIN(st, ids[p.kind]);
  e = cudaLaunchKernelEx(&cfg, expert_rank_kernel, ma, mb, mb2, p);
  NF4_PROF_END(st, ids[p.kind]);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nf4
