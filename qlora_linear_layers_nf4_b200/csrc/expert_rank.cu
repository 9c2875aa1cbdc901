// The rank-r activations of the expert layer on the sm_100a tensor cores:
//   T = s x A_e^T,  U = s dy B_e      out[m, j] for the rows m of every expert
// One tile is 128 rows of an expert by r columns; the reduction runs in steps of
// 64 through a TMA ring and may be split over the CTAs of a cluster, which sum
// their fp32 partials through distributed shared memory in a fixed order.
// U is written as the terms that dA sums (see expert_grad.cu).  Even and odd steps
// have an accumulator each: the tensor core truncates when it adds, and half as many
// additions to smaller sums lose less.
//
// Bound by latency: T of 4096 rows, K 4096, r 64 reads 36 MB in 23.6 us (DRAM 18 %,
// tensor pipe 8 %): setup, a few ring passes a slice, cluster reduction.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_grad.h"
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
using expert::elect_one;
using expert::ring_wait;
using expert::warp_wait;
using expert::unpack2;

constexpr int kRkThreads = 256;    // A loads, B loads, MMA, TMEM; four epilogue warps
constexpr int kRkStages = 4;
constexpr int kRkMaxSlices = 8;    // CTAs of a cluster
constexpr uint32_t kRkABytes = 128 * 128;

struct RankShared {
  uint64_t full[kRkStages];
  uint64_t empty[kRkStages];
  uint64_t accum;
  uint32_t tmem_base;
  uint32_t abort_flag;
  GroupTable groups;
};

// Four consecutive output columns of one row: T, or the terms of U (each what the
// roundings before it left, f16's second one scaled; nothing is left of an infinity,
// whose difference to itself would be NaN).
__device__ __forceinline__ void rank_store4(const RankParams& p, int row, int col, float4 v) {
  const bool f16 = p.f16 != 0;
  const int64_t at = int64_t(row) * p.r + col;
  float u[4] = {v.x * p.scale, v.y * p.scale, v.z * p.scale, v.w * p.scale};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (p.out[i] == nullptr) break;
    const uint2 w = make_uint2(pack2(f16, u[0], u[1]), pack2(f16, u[2], u[3]));
    *reinterpret_cast<uint2*>(p.out[i] + at) = w;
    const float2 a = unpack2(f16, w.x), b = unpack2(f16, w.y);
    const float rounded[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = isfinite(rounded[j]) ? (u[j] - rounded[j]) * p.lo_mul : 0.0f;
  }
}

__global__ void __launch_bounds__(kRkThreads, 1)
    expert_rank_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                       const RankParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = expert::align_1024(smem_raw);
  const uint32_t b_bytes = uint32_t(p.NP) * 128u;
  const uint32_t stage_bytes = kRkABytes + b_bytes;
  RankShared* sh = reinterpret_cast<RankShared*>(smem + kRkStages * stage_bytes);
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
  if (threadIdx.x == 32) {
    tma_prefetch(&tm_a);
    tma_prefetch(&tm_b);
    for (int s = 0; s < kRkStages; ++s) {
      mbar_init(&sh->full[s], 2);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->accum, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 3) {
    tmem_alloc(&sh->tmem_base, uint32_t(p.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  if (int(blockIdx.x) >= sh->groups.tiles[p.E]) {   // the whole cluster
    if (warp == 3) tmem_dealloc(tmem, uint32_t(p.tmem_cols));
    return;
  }
  const int e = expert_of_tile(&sh->groups, p.E, blockIdx.x);
  const int row0 = sh->groups.start[e] + (blockIdx.x - sh->groups.tiles[e]) * 128;
  const int row_end = sh->groups.start[e + 1];
  const int per = (p.red_steps + p.slices - 1) / p.slices;
  const int step0 = min(int(blockIdx.y) * per, p.red_steps);
  const int nsteps = min(step0 + per, p.red_steps) - step0;

  // Loads (warp 0 the A box, warp 1 the B boxes) and MMAs (warp 2) run as whole
  // warps with one elected lane; warps 4..7 are the epilogue.
  if (warp < 2) {
    const bool issue = elect_one();
    int issued = 0, s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < nsteps; ++i) {
      if (!ring_wait(&sh->empty[s], ph, abort_flag, p.status)) break;
      if (issue) {
        uint8_t* a = smem + s * stage_bytes;
        uint8_t* b = a + kRkABytes;
        const int red0 = (step0 + i) * 64;
        if (warp == 0) {
          mbar_arrive_expect_tx(&sh->full[s], kRkABytes);
          tma_load_2d(a, &tm_a, &sh->full[s], red0, row0);
        } else {
          mbar_arrive_expect_tx(&sh->full[s], b_bytes);
          if (p.kind == kRankT) {
            tma_load_3d(b, &tm_b, &sh->full[s], red0, 0, e);
          } else {
            for (int g = 0; g < p.NP / 64; ++g) tma_load_3d(b + g * 8192, &tm_b, &sh->full[s], 64 * g, red0, e);
          }
        }
      }
      __syncwarp();
      ++issued;
      if (++s == kRkStages) {
        s = 0;
        ph ^= 1;
      }
    }
    if (*abort_flag) {   // unwind: wait (bounded) for the copies in flight
      for (int i = max(0, issued - kRkStages); i < issued; ++i) {
        uint32_t none = 0;
        ring_wait(&sh->full[i % kRkStages], (i / kRkStages) & 1, &none, nullptr);
      }
    }
  } else if (warp == 2) {
    const bool issue = elect_one();
    const uint32_t idesc = idesc_f32acc(128, p.NP, false, b_mn, p.f16 != 0);
    const uint32_t b_sub = b_mn ? 2048u >> 4 : 32u >> 4;
    bool ok = true;
    int s = 0, issued = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nsteps; ++i) {
      ok = ring_wait(&sh->full[s], ph, abort_flag, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t a_base = smem_u32(smem + s * stage_bytes);
      const uint64_t adesc = smem_desc_sw128(a_base, 16, 1024);
      const uint64_t bdesc = smem_desc_sw128(a_base + kRkABytes, b_mn ? 8192 : 16, 1024);
      if (issue) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16(tmem + uint32_t(i & 1) * uint32_t(p.NP), adesc + kk * 2, bdesc + kk * b_sub, idesc, (i > 1 || kk > 0) ? 1u : 0u);
        // the last step's commit goes to accum (nobody waits on its stage)
        umma_commit(i + 1 < nsteps ? &sh->empty[s] : &sh->accum);
      }
      __syncwarp();
      ++issued;
      if (++s == kRkStages) {
        s = 0;
        ph ^= 1;
      }
    }
    if (issue && !ok) drain_issued(sh->empty, issued, kRkStages);
    else if (issue && nsteps == 0) mbar_arrive(&sh->accum);
  } else if (warp >= 4) {
    const bool ok = warp_wait(&sh->accum, 0, abort_flag, p.status);
    tc_fence_after();
    const int quad = warp - 4;
    const int prow = quad * 32 + lane;
    const int row = row0 + prow;
    float* dst = reinterpret_cast<float*>(smem) + prow * p.NP;   // parked partial, chunks swizzled by row
    for (int c = 0; c < p.NP / 32; ++c) {
      if (p.slices == 1 && c * 32 >= p.r) break;
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + c * 32, v);
      tmem_ld_wait();
      if (nsteps > 1) {
        uint32_t w[32];
        tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + p.NP + c * 32, w);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
      }
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ok && nsteps > 0)
          f = make_float4(__uint_as_float(v[4 * g]), __uint_as_float(v[4 * g + 1]), __uint_as_float(v[4 * g + 2]),
                          __uint_as_float(v[4 * g + 3]));
        const int col = c * 32 + 4 * g;
        if (p.slices == 1) {
          if (col < p.r && row < row_end) rank_store4(p, row, col, f);
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
      const int cv = i % vec, rr = i / vec;
      const int trow = int(q) * rows_per + rr;
      const uint32_t off = uint32_t((trow * p.NP + 4 * (cv ^ (trow & 7))) * 4);
      float4 part[kRkMaxSlices], acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int sl = 0; sl < kRkMaxSlices; ++sl)   // all on their way before the first is needed
        if (sl < p.slices) part[sl] = ld_shared_cluster_f4(mapa_shared(base + off, uint32_t(sl)));
#pragma unroll
      for (int sl = 0; sl < kRkMaxSlices; ++sl) {
        if (sl >= p.slices) break;
        acc.x += part[sl].x;
        acc.y += part[sl].y;
        acc.z += part[sl].z;
        acc.w += part[sl].w;
      }
      if (row0 + trow < row_end) rank_store4(p, row0 + trow, 4 * cv, acc);
    }
    cluster_sync();
  }
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, uint32_t(p.tmem_cols));
  }
}

PerDeviceOnce g_attr_done;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

bool ExpertRank::prepare(const GroupedArgs& g, RankKind kind, void* out0, void* out1, void* out2, int sms) {
  const LinearArgs& a = g.lin;
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
  p.lo_mul = a.f16 ? kULoMul : 1.0f;
  p.offsets = g.offsets;
  p.out[0] = static_cast<uint16_t*>(out0);
  p.out[1] = static_cast<uint16_t*>(out1);
  p.out[2] = static_cast<uint16_t*>(a.f16 ? nullptr : out2);
  p.status = a.status;
  bool ok;
  if (kind == kRankT) {
    ok = encode_map_2d(&ma, a.x, MapElem::k16, K, M, 64, 128, sw) &&
         encode_map_stack(&mb, a.A, MapElem::k16, K, r, E, 64, uint32_t(p.NP), sw);
    p.red_steps = int(cdiv(a.K, 64));
  } else {
    ok = encode_map_2d(&ma, a.dy, MapElem::k16, N, M, 64, 128, sw) &&
         encode_map_stack(&mb, a.B, MapElem::k16, r, N, E, 64, 64, sw);
    p.red_steps = int(cdiv(a.N, 64));
  }
  if (!ok) return false;
  const int64_t tiles = max_row_tiles(a.M, g.E, 128);
  if (tiles > int64_t(0x7fffffff)) return false;
  // one wave of about two CTAs per SM, four steps a slice at least
  const int64_t cap = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(2 * sms / tiles, kRkMaxSlices), p.red_steps / 4));
  p.slices = 1;
  while (p.slices * 2 <= cap) p.slices *= 2;
  p.tmem_cols = 64;
  while (p.tmem_cols < 2 * p.NP) p.tmem_cols *= 2;
  smem = size_t(kRkStages) * (kRkABytes + size_t(p.NP) * 128) + sizeof(RankShared) + 1024;
  grid = dim3(unsigned(tiles), unsigned(p.slices), 1);
  return true;
}

cudaError_t ExpertRank::run(cudaStream_t st, int* launches) const {
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
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = grid.y;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int id = p.kind == kRankT ? kKGroupedT : kKGroupedU;
  NF4_PROF_BEGIN(st, id);
  e = cudaLaunchKernelEx(&cfg, expert_rank_kernel, ma, mb, p);
  NF4_PROF_END(st, id);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nf4
