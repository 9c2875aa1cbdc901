// Adapter gradients of the expert layer on the sm_100a tensor cores:
//   dB_e = dy^T T  [N, r]      dA_e = U^T x  [r, K]      sums over the expert's rows
//
// A tile is an expert's 128 outputs (rows of dy^T or x^T, MN-major boxes straight
// from the row-major batch) by 64 adapter columns; the reduction walks the
// expert's ragged rows in steps of 64.  Persistent CTAs take the tiles of both
// gradients round robin in one launch; rings and two accumulators run on across
// tiles, so that an expert with a handful of rows costs its loads and not a
// kernel's start.
//
// TMA boxes start at any row, so only a tile's last step holds rows of the next
// expert.  Its MMAs stop at the next multiple of 16 rows, and a warp clears the up
// to 15 rows between in both operands (a cleared row times NaN would still be NaN)
// as soon as they land, ahead of the MMAs.
//
// dA sums products of U, whose rounding to 16 bits would be its largest error by
// far (2^-9 against 2^-24 for a sum's step).  U comes as three bf16 terms that
// together hold its 24 bits, or as two f16 terms, the second scaled by 2^11 (its
// values would be subnormal otherwise).  They cost adapter columns in a product that
// is bound by reading x.  The tensor core truncates when it adds to an accumulator,
// so what counts is how often it adds to a large one: the first terms of even and
// odd steps have an accumulator each and the small terms a third, summed in fp32 at
// the end (dA's error on 512 rows an expert: 2.0e-6 with one, 0.5e-6 with three).
//
// 4096 rows of 4 experts of 4096 x 4096, r 64: 33 us for 73 MB (DRAM 27 %, tensor
// pipe 21 %); 64 experts of 1024 x 2048 with 4,001 uneven rows: 29 us.  Bound by the
// steps' latency and by the CTAs that drew the longest tiles.
#include <algorithm>

#include <cuda.h>
#include <cuda_runtime.h>

#include "expert_grad.h"
#include "grouped.cuh"
#include "kernels.h"
#include "nf4_common.cuh"
#include "ring_wait.cuh"
#include "tc_common.cuh"
#include "tensor_maps.h"

namespace nf4 {
namespace {

using namespace tc;
using expert::elect_one;
using expert::ring_wait;
using expert::warp_wait;

constexpr int kGrThreads = 256;    // A loads, B loads, MMA, tail rows; four epilogue warps
constexpr int kGrCols = 64;        // adapter columns per tile
constexpr int kGrMaxStages = 6;
constexpr uint32_t kGrABytes = 128 * 128;

struct GradShared {
  uint64_t full[kGrMaxStages];
  uint64_t empty[kGrMaxStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t fixed[kGrMaxStages];   // the rows past the expert in a tile's last step are cleared
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
  GroupTable groups;
};

struct GradTile {
  int job;             // 0: dA, 1: dB
  int e, row0, col0;   // expert, first output row, first adapter column
  int tok0, cnt;       // the expert's rows
};
__device__ __forceinline__ GradTile grad_tile(const GroupTable* g, const GradParams& p, int id) {
  GradTile t;
  t.job = id >= p.job[0].tiles ? 1 : 0;
  if (t.job) id -= p.job[0].tiles;
  const int rt = p.job[t.job].row_tiles, per = rt * p.col_tiles;
  t.e = id / per;
  const int q = id - t.e * per, c = q / rt;
  t.col0 = c * kGrCols;
  t.row0 = (q - c * rt) * 128;
  t.tok0 = g->start[t.e];
  t.cnt = g->start[t.e + 1] - t.tok0;
  return t;
}

__global__ void __launch_bounds__(kGrThreads, 1)
    expert_grad_kernel(const __grid_constant__ GradMaps maps, const GradParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = expert::align_1024(smem_raw);
  const uint32_t stage_bytes = p.stage_bytes;
  GradShared* sh = reinterpret_cast<GradShared*>(smem + p.stages * stage_bytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sh->abort_flag;
  const int tiles = p.job[0].tiles + p.job[1].tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&sh->full[s], 2);
      mbar_init(&sh->empty[s], 2);   // the MMAs and the tail warp
      mbar_init(&sh->fixed[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], 4);
    }
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch(&maps.a[0]);
    tma_prefetch(&maps.b[0]);
  }
  if (warp == 3) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 4) build_groups(&sh->groups, p.offsets, p.E, p.M, 64, blockIdx.x == 0 ? p.status : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (warp < 2) {
    // ---------------- loads: warp 0 the A boxes, warp 1 the adapter terms, [64
    // rows][128 bytes] one after another
    const bool issue = elect_one();
    int s = 0, issued = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
      const GradTile t = grad_tile(&sh->groups, p, id);
      const GradJob& job = p.job[t.job];
      for (int k = 0; k < t.cnt; k += 64) {
        ok = ring_wait(&sh->empty[s], ph, abort_flag, p.status);
        if (!ok) break;
        if (issue) {
          uint8_t* a = smem + s * stage_bytes;
          if (warp == 0) {
            mbar_arrive_expect_tx(&sh->full[s], kGrABytes);
            if (job.whole) {
              tma_load_3d(a, &maps.a[t.job], &sh->full[s], 0, t.tok0 + k, t.row0 / 64);
            } else {
              tma_load_2d(a, &maps.a[t.job], &sh->full[s], t.row0, t.tok0 + k);
              tma_load_2d(a + 8192, &maps.a[t.job], &sh->full[s], t.row0 + 64, t.tok0 + k);
            }
          } else {
            mbar_arrive_expect_tx(&sh->full[s], uint32_t(job.terms) * 8192u);
            tma_load_3d(a + kGrABytes, &maps.b[t.job], &sh->full[s], t.col0, t.tok0 + k, 0);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == p.stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (*abort_flag)   // unwind: wait (bounded) for the copies in flight
      for (int j = max(0, issued - p.stages); j < issued; ++j) {
        uint32_t none = 0;
        ring_wait(&sh->full[j % p.stages], (j / p.stages) & 1, &none, nullptr);
      }
  } else if (warp == 2) {
    // ---------------- MMA: the whole warp walks the steps, one lane issues
    const bool issue = elect_one();
    int s = 0, n = 0;
    uint32_t ph = 0, fixed_ph = 0;   // fixed_ph: bit s for stage s
    bool ok = true;
    for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
      const GradTile t = grad_tile(&sh->groups, p, id);
      if (t.cnt == 0) continue;   // the epilogue writes zeros
      const int terms = p.job[t.job].terms;
      const int cols = min(kGrCols, (p.r - t.col0 + 15) & ~15);
      const uint32_t idesc = idesc_f32acc(128, cols, true, true, p.f16 != 0);
      const uint32_t d = tmem + uint32_t(n & 1) * 256u;
      ok = ring_wait(&sh->acc_empty[n & 1], ((n >> 1) & 1) ^ 1, abort_flag, p.status);
      if (!ok) break;
      for (int k = 0; k < t.cnt; k += 64) {
        ok = ring_wait(&sh->full[s], ph, abort_flag, p.status);
        const int left = t.cnt - k;
        if (ok && left < 64 && (left & 15)) {
          ok = ring_wait(&sh->fixed[s], (fixed_ph >> s) & 1u, abort_flag, p.status);
          fixed_ph ^= 1u << s;
        }
        if (!ok) break;
        tc_fence_after();
        const uint32_t a_base = smem_u32(smem + s * stage_bytes);
        const uint64_t adesc = smem_desc_sw128(a_base, 8192, 1024);
        const uint64_t bdesc = smem_desc_sw128(a_base + kGrABytes, 8192, 1024);
        if (issue) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk * 16 >= left) break;
            // first terms: columns 0 (even steps) and 64 (odd); the others: 128
            const uint32_t first = (k >> 6) & 1;
            umma_f16(d + 64u * first, adesc + kk * 128, bdesc + kk * 128, idesc, (k >= 128 || kk > 0) ? 1u : 0u);
            if (terms > 1) umma_f16(d + 128u, adesc + kk * 128, bdesc + 512 + kk * 128, idesc, (k > 0 || kk > 0) ? 1u : 0u);
            if (terms > 2) umma_f16(d + 128u, adesc + kk * 128, bdesc + 1024 + kk * 128, idesc, 1u);
          }
          umma_commit(&sh->empty[s]);
          if (k + 64 >= t.cnt) umma_commit(&sh->acc_full[n & 1]);
        }
        __syncwarp();
        if (++s == p.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      ++n;
    }
    if (!ok && issue) {   // unwind: wait (bounded) for the MMAs in flight
      umma_commit(&sh->drain);
      uint32_t none = 0;
      ring_wait(&sh->drain, 0, &none, nullptr);
    }
  } else if (warp == 3) {
    // ---------------- tail: clears the rows past an expert's last, up to the next
    // multiple of 16, as soon as a tile's last step has landed.  It walks every
    // step and gives each stage back too, so that it stays within the ring.
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
      const GradTile t = grad_tile(&sh->groups, p, id);
      for (int k = 0; k < t.cnt; k += 64) {
        ok = warp_wait(&sh->full[s], ph, abort_flag, p.status);
        if (!ok) break;
        const int left = t.cnt - k;
        const bool clear = left < 64 && (left & 15);
        if (clear) {
          uint8_t* a = smem + s * stage_bytes;
          const int blocks = 2 + p.job[t.job].terms;   // [64 rows][128 bytes] each, A then the terms
          const int chunks = (16 - (left & 15)) * 8;
          for (int b = 0; b < blocks; ++b)
            for (int i = lane; i < chunks; i += 32)
              *reinterpret_cast<uint4*>(a + b * 8192 + left * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          if (clear) mbar_arrive(&sh->fixed[s]);
          mbar_arrive(&sh->empty[s]);
        }
        if (++s == p.stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
  } else {
    // ---------------- epilogue: lane = output row, register = adapter column
    const int quad = warp - 4;
    int n = 0;
    for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
      const GradTile t = grad_tile(&sh->groups, p, id);
      const GradJob& job = p.job[t.job];
      const int b = n & 1;
      if (t.cnt > 0) {
        if (!warp_wait<100>(&sh->acc_full[b], (n >> 1) & 1, abort_flag, p.status)) break;
        ++n;
        tc_fence_after();
      }
      const int row = t.row0 + quad * 32 + lane;
      const int cols = min(kGrCols, p.r - t.col0);
      for (int c = 0; c < cols; c += 32) {
        float f[32];
        if (t.cnt > 0) {
          const uint32_t at = tmem + (uint32_t(quad * 32) << 16) + uint32_t(b) * 256u + c;
          uint32_t v[32];
          tmem_ld_32x32b_x32(at, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
          if (t.cnt > 64) {
            tmem_ld_32x32b_x32(at + 64u, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] += __uint_as_float(v[i]);
          }
          if (job.terms > 1) {
            tmem_ld_32x32b_x32(at + 128u, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = fmaf(__uint_as_float(v[i]), p.lo_scale, f[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = 0.0f;
        }
        if (row >= job.Mo) continue;
        if (t.job == 0) {     // dA: [r, K] of the expert
          float* o = job.out + (int64_t(t.e) * p.r + t.col0 + c) * job.Mo + row;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < cols) o[int64_t(i) * job.Mo] = f[i];
        } else {              // dB: [N, r] of the expert
          float* o = job.out + (int64_t(t.e) * job.Mo + row) * p.r + t.col0 + c;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            if (c + i < cols) *reinterpret_cast<float4*>(o + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
        }
      }
      if (t.cnt > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->acc_empty[b]);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

PerDeviceOnce g_attr_done;

}  // namespace

bool ExpertGrad::prepare(const GroupedArgs& g, const void* T, const void* U, int u_terms, int sms) {
  const LinearArgs& a = g.lin;
  const uint64_t M = uint64_t(a.M), r = uint64_t(a.r);
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  p = GradParams{};
  p.E = g.E;
  p.M = int(a.M);
  p.r = a.r;
  p.f16 = a.f16;
  p.lo_scale = a.f16 ? 1.0f / kULoMul : 1.0f;
  p.offsets = g.offsets;
  p.status = a.status;
  p.col_tiles = (a.r + kGrCols - 1) / kGrCols;
  const void* in[2] = {a.x, a.dy};
  const void* terms[2] = {U, T};
  bool ok = true;
  int64_t tiles = 0;
  for (int i = 0; i < 2; ++i) {
    GradJob& j = p.job[i];
    j.Mo = int(i == 0 ? a.K : a.N);
    j.out = i == 0 ? a.dA : a.dB;
    j.terms = i == 0 ? u_terms : 1;
    j.row_tiles = (j.Mo + 127) / 128;
    const int64_t n = int64_t(j.row_tiles) * p.col_tiles * g.E;
    tiles += n;
    if (tiles > int64_t(0x7fffffff)) return false;
    j.tiles = int(n);
    // Whole 64-column groups: both of a tile in one box, as [group][row][64].
    j.whole = j.Mo % 64 == 0;
    const uint64_t Mo = uint64_t(j.Mo);
    if (j.whole) {
      const uint64_t dims[3] = {64, M, Mo / 64}, strides[2] = {Mo * 2, 128};
      const uint32_t box[3] = {64, 64, 2};
      ok = ok && encode_map(&maps.a[i], in[i], MapElem::k16, 3, dims, strides, box, sw);
    } else {
      ok = ok && encode_map_2d(&maps.a[i], in[i], MapElem::k16, Mo, M, 64, 64, sw);
    }
    const uint64_t dims[3] = {r, M, uint64_t(j.terms)}, strides[2] = {r * 2, M * r * 2};
    const uint32_t box[3] = {64, 64, uint32_t(j.terms)};
    ok = ok && encode_map(&maps.b[i], terms[i], MapElem::k16, 3, dims, strides, box, sw);
  }
  p.stage_bytes = kGrABytes + 8192u * uint32_t(u_terms);
  p.stages = int(std::min<uint32_t>(kGrMaxStages, 208u * 1024u / p.stage_bytes));
  smem = size_t(p.stages) * p.stage_bytes + sizeof(GradShared) + 1024;
  grid = unsigned(std::min<int64_t>(tiles, sms));
  return ok;
}

cudaError_t ExpertGrad::run(cudaStream_t st, int* launches) const {
  const int dev = PerDeviceOnce::current();
  cudaError_t e = cudaSuccess;
  if (!g_attr_done.done(dev)) {
    e = cudaFuncSetAttribute(expert_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e != cudaSuccess) return e;
    g_attr_done.mark(dev);
  }
  NF4_PROF_BEGIN(st, kKGroupedGrad);
  expert_grad_kernel<<<grid, kGrThreads, smem, st>>>(maps, p);
  NF4_PROF_END(st, kKGroupedGrad);
  e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nf4
