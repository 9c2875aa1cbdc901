// The 8-bit floating point linear on the sm_100a tensor cores:
//   y[m, n] = sum_b sx[m, b] sw[n / 128, b] (sum_{k in block b} wq[n, k] xq[m, k]) (+ bias[n])
//
// Tokens on the TMEM lanes (A), weight rows as N (B), both K-major e4m3 by TMA; a ring stage
// is one block of 128 along K, four kind::f8f6f4 MMAs.  The scales change from block to
// block, so the MMAs of a block start a fresh accumulator, one of two that alternate, and
// the epilogue warps add it to fp32 sums in registers, one FMA an element with the product
// of the two scales: a lane is a token and the columns of a warp lie in one weight block, so
// that product is one number per thread and block.
//
// Wide tiles are 256 x 256 by a pair of CTAs (cta_group::2): the MMAs of a block take 512
// cycles, reading the accumulator (128 x 256 of it in each CTA) 256 and the FMAs 256, on
// eight warps of 128 columns each.  Where such tiles would leave SMs idle, a CTA takes
// 128 x 128, 64 or 32, and the blocks along K may be shared by a cluster of CTAs, which add
// their fp32 sums through distributed shared memory in their order.
// Roles: warp 0 token TMA, warp 1 weight TMA, warp 2 MMA (the pair's leader issues), from
// warp 4 on the sums.  Output in pieces of 32 rows of 64 bytes through shared memory by TMA.
//
// 4,096 tokens through 11008 x 4096 take 168 us (2.2 PFLOP/s, tensor pipe 53 % active; without
// the sums 132, at the power limit).  The bound is the chain of a block over two accumulators:
// 512 cycles of MMAs, 230 until their end is seen, 490 to add 128 columns a warp, 290 until the
// MMAs may start again.  Sixteen warps of 64 columns, scales from a ring in shared memory and
// halves of 128 columns were slower (192, 185 and 177 us or more).
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8.h"
#include "nf4_common.cuh"
#include "nf4_dequant.cuh"
#include "pair_tile.cuh"
#include "ring_wait.cuh"
#include "tc_common.cuh"
#include "tensor_maps.h"

namespace nf4 {
namespace {

using namespace tc;
using namespace expert;

constexpr int kEpiWarp = 4;
constexpr uint32_t kXBytes = 128 * 128;
constexpr int kMaxParts = kFp8MaxParts;
constexpr uint32_t kPiece = 2048;        // of a warp: 32 rows of 64 bytes of the result

template <int NT>
struct Cfg {
  static constexpr int kPair = NT == 256 ? 2 : 1;                 // CTAs of a tile
  static constexpr int kRows = 128 * kPair;                       // tokens of a tile
  static constexpr int kCols = NT > 128 ? 128 : NT;               // columns of a warp
  static constexpr int kEpiWarps = 4 * NT / kCols;
  static constexpr int kThreads = 32 * (kEpiWarp + kEpiWarps);
  static constexpr uint32_t kWBytes = uint32_t(NT / kPair) * 128;
  static constexpr uint32_t kStage = kXBytes + kWBytes;
  static constexpr int kStages = 6;
  static constexpr uint32_t kTmem = NT == 256 ? 512 : 2 * NT;
};

struct Fp8Shared {
  uint64_t full[6];
  uint64_t empty[6];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
};
template <int NT>
constexpr size_t fp8_smem() {
  return size_t(Cfg<NT>::kStages) * Cfg<NT>::kStage + Cfg<NT>::kEpiWarps * kPiece + sizeof(Fp8Shared) + 1024;
}
static_assert(fp8_smem<256>() <= 232448, "shared memory of one CTA");

// The wait of a whole warp, every lane polling: a poll that succeeds at once costs no shuffle.
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, abort_flag, status);
}

// acc + v * scale of two columns in one instruction.
__device__ __forceinline__ void add2(float2& acc, uint32_t v0, uint32_t v1, float2 scale) {
  uint64_t a, v, s;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(acc.x), "f"(acc.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(s) : "f"(scale.x), "f"(scale.y));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(v), "l"(s));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(acc.x), "=f"(acc.y) : "l"(a));
}

// e4m3 x e4m3 -> fp32 (kind::f8f6f4, both K-major).
template <int PAIR>
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  if (PAIR == 2) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
constexpr uint32_t idesc_e4m3(int M, int N) { return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24); }

// Element of a parked tile [128][NT]: 16-byte chunks swizzled by row.
template <int NT>
__device__ __forceinline__ int park_at(int row, int col) {
  return row * NT + 4 * ((col >> 2) ^ (row & 7)) + (col & 3);
}

__device__ __forceinline__ float bias_of(const Fp8Params& p, int col) {
  const int at = min(col, p.N - 1);
  return p.dtype == NF4_F32   ? __ldg(static_cast<const float*>(p.bias) + at)
         : p.dtype == NF4_F16 ? __half2float(static_cast<const __half*>(p.bias)[at])
                              : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[at]);
}

// The parts of a tile added up in their order, each CTA of the cluster a share of the rows.
// All threads; the second barrier keeps the parts alive.
template <int NT>
__device__ __forceinline__ void join_parts(const Fp8Params& p, const float* park, int parts, int id) {
  cluster_sync();
  const int q = int(cluster_ctarank());
  const int ct = id / p.row_tiles, rt = id - ct * p.row_tiles;
  const int rows = min(128, p.M - rt * 128), r0 = rows * q / parts, r1 = rows * (q + 1) / parts;
  constexpr int kVec = NT / 4;
  const uint32_t base = smem_u32(park);
  for (int i = threadIdx.x; i < (r1 - r0) * kVec; i += blockDim.x) {
    const int row = r0 + i / kVec, c = 4 * (i % kVec), col = ct * NT + c;
    float4 part[kMaxParts], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kMaxParts; ++s)   // all on their way before the first is needed
      if (s < parts) part[s] = ld_shared_cluster_f4(mapa_shared(base + uint32_t(park_at<NT>(row, c)) * 4u, uint32_t(s)));
#pragma unroll
    for (int s = 0; s < kMaxParts; ++s) {
      if (s >= parts) break;
      v.x += part[s].x;
      v.y += part[s].y;
      v.z += part[s].z;
      v.w += part[s].w;
    }
    if (col >= p.N) continue;
    if (p.bias != nullptr)
      v = make_float4(v.x + bias_of(p, col), v.y + bias_of(p, col + 1), v.z + bias_of(p, col + 2), v.w + bias_of(p, col + 3));
    const int64_t at = int64_t(rt * 128 + row) * p.N + col;
    if (p.dtype == NF4_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = v;
    } else {
      const bool f16 = p.dtype == NF4_F16;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) = make_uint2(pack2(f16, v.x, v.y), pack2(f16, v.z, v.w));
    }
  }
  cluster_sync();
}

template <int NT>
__device__ __forceinline__ void fp8_gemm_body(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& my, const Fp8Params& p) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = expert::align_1024(smem_raw);
  uint8_t* out_base = smem + C::kStages * C::kStage;
  Fp8Shared* sh = reinterpret_cast<Fp8Shared*>(out_base + C::kEpiWarps * kPiece);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = C::kPair == 2 ? cluster_ctarank() : 0u;
  volatile uint32_t* abort_flag = &sh->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], C::kEpiWarps * C::kPair);   // leader: both CTAs' warps
    }
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch(&mx);
    tma_prefetch(&mw);
    tma_prefetch(&my);
  }
  if (warp == 2) {
    if (C::kPair == 2) {
      tmem_alloc_pair(&sh->tmem_base, C::kTmem);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&sh->tmem_base, C::kTmem);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (C::kPair == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int first = int(blockIdx.x) / C::kPair, step = int(gridDim.x) / C::kPair;
  // Blocks of this CTA: all, or (one tile a CTA) its part of them; the parts' sums are joined.
  const int parts = C::kPair == 2 ? 1 : int(gridDim.y);
  const int b0 = parts == 1 ? 0 : p.kb * int(blockIdx.y) / parts, b1 = parts == 1 ? p.kb : p.kb * (int(blockIdx.y) + 1) / parts;
  auto leader_bar = [&](uint64_t* bar) { return C::kPair == 2 ? mapa_shared(smem_u32(bar), 0) : smem_u32(bar); };
  grid_dep_wait();
  // The sums of wide tiles want more registers than an even split gives: 4 warps x 56 + 8 x 224,
  // the 12 x 168 that the CTA was launched with.
  auto few_registers = [] {
    if constexpr (NT == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  };

  if (warp < 2) {
    // ---------------- TMA: tokens (warp 0, which expects every byte of a stage) and weight
    few_registers();
    const bool issue = elect_one();
    bool ok = true;
    int s = 0, issued = 0;
    uint32_t ph = 1;
    for (int id = first; id < p.tiles && ok; id += step) {
      const int ct = id / p.row_tiles, rt = id - ct * p.row_tiles;
      const int y = warp == 0 ? rt * C::kRows + 128 * int(rank) : ct * NT + (NT / C::kPair) * int(rank);
      for (int b = b0; b < b1; ++b) {
        ok = ring_wait(&sh->empty[s], ph, abort_flag, p.status);
        if (!ok) break;
        if (issue) {
          uint8_t* dst = smem + s * C::kStage + (warp == 0 ? 0u : kXBytes);
          if (warp == 0 && rank == 0) mbar_arrive_expect_tx(&sh->full[s], C::kPair * (p.x_bytes + C::kWBytes));
          if (C::kPair == 2) tma_load_2d_pair(dst, warp == 0 ? &mx : &mw, leader_bar(&sh->full[s]), b * 128, y);
          else tma_load_2d(dst, warp == 0 ? &mx : &mw, &sh->full[s], b * 128, y);
        }
        __syncwarp();
        ++issued;
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (*abort_flag)   // unwind: wait (bounded) for the stages in flight
      for (int j = max(0, issued - C::kStages); j < issued; ++j) {
        uint32_t none = 0;
        ring_wait(&sh->empty[j % C::kStages], (j / C::kStages) & 1, &none, nullptr);
      }
  } else if (warp == 2) {
    // ---------------- MMA
    few_registers();
    if (rank == 0) {
      const bool issue = elect_one();
      const uint64_t x_desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t w_desc = smem_desc_sw128(smem_u32(smem) + kXBytes, 16, 1024);
      constexpr uint32_t idesc = idesc_e4m3(C::kRows, NT);
      bool ok = true;
      int s = 0, n = 0;
      uint32_t ph = 0;
      for (int id = first; id < p.tiles && ok; id += step) {
        for (int b = b0; b < b1; ++b, ++n) {
          ok = mbar_wait_cluster(&sh->full[s], ph, abort_flag, p.status);
          if (ok) ok = mbar_wait_cluster(&sh->acc_empty[n & 1], ((n >> 1) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          if (issue) {
            const uint32_t d = tmem + uint32_t(n & 1) * uint32_t(NT);
            const uint32_t at = uint32_t(s) * (C::kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma_f8<C::kPair>(d, x_desc + at + kk * 2, w_desc + at + kk * 2, idesc, kk > 0 ? 1u : 0u);
            // one commit a block: the warps that read the accumulator give the stage back
            if (C::kPair == 2) umma_commit_pair_mc(&sh->acc_full[n & 1], 0x3);
            else umma_commit(&sh->acc_full[n & 1]);
          }
          __syncwarp();
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok && issue) {   // unwind: wait (bounded) for the MMAs in flight
        if (C::kPair == 2) umma_commit_pair_mc(&sh->drain, 0x1);
        else umma_commit(&sh->drain);
        uint32_t none = 0;
        ring_wait(&sh->drain, 0, &none, nullptr);
      }
    }
  } else if (warp == 3) {
    few_registers();
  } else {
    // ---------------- sums: lane = token, C::kCols columns a warp
    if constexpr (NT == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int quad = warp & 3, group = (warp - kEpiWarp) >> 2;   // TMEM lanes; columns
    uint8_t* buf = out_base + (warp - kEpiWarp) * kPiece;
    int s = 0, n = 0;
    bool ok = true;
    for (int id = first; id < p.tiles && ok; id += step) {
      const int ct = id / p.row_tiles, rt = id - ct * p.row_tiles;
      const int row0 = rt * C::kRows + 128 * int(rank) + quad * 32, col0 = ct * NT + group * C::kCols;
      const float* sx = p.x_scale + int64_t(min(row0 + lane, p.M - 1)) * p.kb;
      const float* sw = p.w_scale + int64_t(min(col0, p.N - 1) / 128) * p.kb;
      float nx = __ldg(sx + b0), nw = __ldg(sw + b0);
      float2 acc[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      for (int b = b0; b < b1; ++b, ++n) {
        ok = all_wait(&sh->acc_full[n & 1], (n >> 1) & 1, abort_flag, p.status);
        if (!ok) break;
        if (warp == kEpiWarp + C::kEpiWarps - 1 && lane == 0) mbar_arrive(&sh->empty[s]);
        if (++s == C::kStages) s = 0;
        tc_fence_after();
        const uint32_t at = tmem + (uint32_t(quad * 32) << 16) + uint32_t(n & 1) * uint32_t(NT) + group * C::kCols;
        const float2 scale = make_float2(nx * nw, nx * nw);   // loaded a block ahead
        const int nb = min(b + 1, b1 - 1);
        nx = __ldg(sx + nb);
        nw = __ldg(sw + nb);
        // 32 columns are on their way while the 32 before are added
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(at, v[0]);
#pragma unroll
        for (int c = 0; c < C::kCols / 32; ++c) {
          tmem_ld_wait();
          if (c + 1 < C::kCols / 32) {
            tmem_ld_32x32b_x32(at + 32 * (c + 1), v[(c + 1) & 1]);
          } else {   // every column is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (C::kPair == 2) arrive_leader(leader_bar(&sh->acc_empty[n & 1]));
              else mbar_arrive(&sh->acc_empty[n & 1]);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) add2(acc[16 * c + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], scale);
        }
      }
      if (!ok) break;
      if (C::kPair == 1 && parts > 1) {   // for the other CTAs: the ring is done with
        float* park = reinterpret_cast<float*>(smem);
        const int row = quad * 32 + lane;
#pragma unroll
        for (int c = 0; c < C::kCols; c += 4)
          *reinterpret_cast<float4*>(park + park_at<NT>(row, group * C::kCols + c)) =
              make_float4(acc[c / 2].x, acc[c / 2].y, acc[c / 2 + 1].x, acc[c / 2 + 1].y);
        break;
      }
      // ---- bias, rounding; pieces of 32 rows x 64 bytes through shared memory (64-byte
      // swizzle: chunk j at j ^ ((row >> 1) & 3))
      if (p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < C::kCols / 2; ++i) {
          acc[i].x += bias_of(p, col0 + 2 * i);
          acc[i].y += bias_of(p, col0 + 2 * i + 1);
        }
      }
      auto piece = [&](int col, const uint4 (&chunk)[4]) {
        if (lane == 0) bulk_wait_group_read<0>();   // the store before has read the piece
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = chunk[j];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&my, buf, col, row0);   // rows past M, columns past N: clipped
          bulk_commit_group();
        }
      };
      if (p.dtype == NF4_F32) {
#pragma unroll
        for (int c = 0; c < C::kCols; c += 16) {
          if (col0 + c >= p.N || row0 >= p.M) break;
          uint4 chunk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            chunk[j] = make_uint4(__float_as_uint(acc[c / 2 + 2 * j].x), __float_as_uint(acc[c / 2 + 2 * j].y),
                                  __float_as_uint(acc[c / 2 + 2 * j + 1].x), __float_as_uint(acc[c / 2 + 2 * j + 1].y));
          piece(col0 + c, chunk);
        }
      } else {
        const bool f16 = p.dtype == NF4_F16;
#pragma unroll
        for (int c = 0; c < C::kCols; c += 32) {
          if (col0 + c >= p.N || row0 >= p.M) break;
          uint4 chunk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            chunk[j] = make_uint4(pack2(f16, acc[c / 2 + 4 * j].x, acc[c / 2 + 4 * j].y),
                                  pack2(f16, acc[c / 2 + 4 * j + 1].x, acc[c / 2 + 4 * j + 1].y),
                                  pack2(f16, acc[c / 2 + 4 * j + 2].x, acc[c / 2 + 4 * j + 2].y),
                                  pack2(f16, acc[c / 2 + 4 * j + 3].x, acc[c / 2 + 4 * j + 3].y));
          piece(col0 + c, chunk);
        }
      }
    }
    if (lane == 0) bulk_wait_group_all();
  }

  __syncwarp();
  tc_fence_before();
  if (C::kPair == 2) cluster_sync();
  else __syncthreads();
  if (C::kPair == 1 && parts > 1) join_parts<NT>(p, reinterpret_cast<const float*>(smem), parts, first);
  if (warp == 2) {
    tc_fence_after();
    if (C::kPair == 2) tmem_dealloc_pair(tmem, C::kTmem);
    else tmem_dealloc(tmem, C::kTmem);
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<256>::kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                    const __grid_constant__ CUtensorMap my, const Fp8Params p) {
  fp8_gemm_body<256>(mx, mw, my, p);
}
template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 1)
    fp8_tile_gemm_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                         const __grid_constant__ CUtensorMap my, const Fp8Params p) {
  fp8_gemm_body<NT>(mx, mw, my, p);
}

PerDeviceOnce g_attr_done;

cudaError_t set_attrs() {
  const int dev = PerDeviceOnce::current();
  if (g_attr_done.done(dev)) return cudaSuccess;
  const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(fp8_pair_kernel, attr, int(fp8_smem<256>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_tile_gemm_kernel<128>, attr, int(fp8_smem<128>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_tile_gemm_kernel<64>, attr, int(fp8_smem<64>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_tile_gemm_kernel<32>, attr, int(fp8_smem<32>()));
  if (e == cudaSuccess) g_attr_done.mark(dev);
  return e;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

bool Fp8Gemm::prepare(const Fp8LinearArgs& a, int sms) {
  const uint64_t M = uint64_t(a.M), N = uint64_t(a.N), K = uint64_t(a.K);
  const Fp8GemmPlan plan = fp8_gemm_plan(a.M, a.N, a.K, sms);
  tile_n = plan.tile_n;
  parts = plan.parts;
  const int pair = tile_n == 256 ? 2 : 1;
  // Few tokens: a box of as many rows (the other lanes' results are never stored).  With
  // fewer than 32 tokens in boxes of 128 rows 4096 x 4096 took 18 us against 11.4 with 33.
  const int x_rows = a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
  const CUtensorMapSwizzle s128 = CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = encode_map_2d(&mx, a.x, MapElem::kU8, K, M, 128, uint32_t(x_rows), s128) &&
            encode_map_2d(&mw, a.w, MapElem::kU8, K, N, 128, uint32_t(tile_n / pair), s128);
  const uint32_t rows = uint32_t(std::min<uint64_t>(M, 32));
  ok = ok && (a.dtype == NF4_F32 ? make_map_2d_f32(&my, a.y, N, M, 16, rows, CU_TENSOR_MAP_SWIZZLE_64B)
                                 : encode_map_2d(&my, a.y, MapElem::k16, N, M, 32, rows, CU_TENSOR_MAP_SWIZZLE_64B));
  p = Fp8Params{};
  p.M = int(a.M);
  p.N = int(a.N);
  p.kb = int(cdiv(a.K, kFp8Block));
  p.row_tiles = int(cdiv(a.M, 128 * pair));
  const int64_t tiles = int64_t(p.row_tiles) * cdiv(a.N, tile_n);
  p.tiles = int(tiles);
  p.x_bytes = uint32_t(x_rows) * 128u;
  p.dtype = a.dtype;
  p.w_scale = a.w_scale;
  p.x_scale = a.x_scale;
  p.bias = a.bias;
  p.y = a.y;
  p.status = a.status;
  grid = unsigned(parts > 1 ? tiles : pair * std::min<int64_t>(tiles, std::max(sms / pair, 1)));   // parts: a tile a CTA
  return ok && tiles <= int64_t(0x7fffffff);
}

cudaError_t Fp8Gemm::run(cudaStream_t st, int* launches) const {
  cudaError_t e = set_attrs();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, unsigned(parts), 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int attrs = 0;
  if (parts > 1) {
    attr[attrs].id = cudaLaunchAttributeClusterDimension;
    attr[attrs].val.clusterDim.x = 1;
    attr[attrs].val.clusterDim.y = unsigned(parts);
    attr[attrs++].val.clusterDim.z = 1;
  }
  attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[attrs].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(prof_on() ? attrs : attrs + 1);
  NF4_PROF_BEGIN(st, kKFp8Linear);
  auto go = [&](auto kernel, int threads, size_t smem) {
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, kernel, mx, mw, my, p);
  };
  e = tile_n == 256   ? go(fp8_pair_kernel, Cfg<256>::kThreads, fp8_smem<256>())
      : tile_n == 128 ? go(fp8_tile_gemm_kernel<128>, Cfg<128>::kThreads, fp8_smem<128>())
      : tile_n == 64  ? go(fp8_tile_gemm_kernel<64>, Cfg<64>::kThreads, fp8_smem<64>())
                      : go(fp8_tile_gemm_kernel<32>, Cfg<32>::kThreads, fp8_smem<32>());
  NF4_PROF_END(st, kKFp8Linear);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nf4
