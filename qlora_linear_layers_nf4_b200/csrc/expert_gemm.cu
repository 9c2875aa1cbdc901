// The big products of the expert layer and of the 8-bit linear on the sm_100a
// tensor cores, rows sorted by expert:
//   kFwd   y[m, n]  = sum_k W'_e[n, k] x[m, k] + sum_j B_e[n, j] T[m, j] (+ bias_e[n])
//   kDx    dx[m, k] = sum_n W'_e[n, k] dy[m, n] + sum_j A_e[j, k] U[m, j]
//   kI8    y[m, n]  = (sum_k wq[n, k] xq[m, k]) sx[m] sw[n] (+ bias[n])
//
// The weight is the A operand of the MMA (128 outputs of an expert = the 128
// TMEM lanes) and the tokens are the B operand, whose count is any multiple of
// 16 up to 256: an expert's ragged rows are cut into even tiles that waste at
// most 15 columns, where tokens on the lanes would waste up to 127.  It also
// puts the outputs' contiguous dimension on the lanes, so a row's results are
// stored under its own row predicate, rows of other experts untouched.
//
// One persistent CTA per SM walks over (expert, 128 outputs, token tile); the
// tile list comes from the offsets in device memory, scanned once per CTA.
// Roles: two token-tile TMA producers, one producer of the weight side (NF4
// code boxes or the int8 tile), one MMA issuer, four epilogue warps, eight
// dequant warps (NF4).  Rings: four stages of [weight tile 16 KB | token tile
// 32 KB], three code boxes of two K steps; two accumulators of 256 TMEM
// columns, so a tile's epilogue runs under the next tile's MMAs.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_gemm.h"
#include "grouped.cuh"
#include "kernels.h"
#include "nf4_common.cuh"
#include "nf4_dequant.cuh"
#include "tc_common.cuh"
#include "tensor_maps.h"

namespace nf4 {
namespace {

using namespace tc;
using namespace expert;

constexpr int kFwd = 0;
constexpr int kDx = 1;
constexpr int kI8 = 2;

constexpr int kTileW = 128;                 // outputs per tile
constexpr int kTileT = 256;                 // tokens per tile at most
constexpr int kStages = 4;
constexpr uint32_t kWBytes = 128 * 128;     // weight tile: 128 x 128 bytes
constexpr uint32_t kTBytes = 256 * 128;     // token tile
constexpr uint32_t kStageBytes = kWBytes + kTBytes;
constexpr int kCodeSteps = 2;               // K steps per code box
constexpr int kCodeSlots = 3;
constexpr uint32_t kCodeBytes = 128 * 64;
constexpr int kDeqWarps = 8;
constexpr int kEpiWarp = 4;                 // warps 4..7
constexpr int kDeqWarp = 8;                 // warps 8..15

struct GemmShared {
  uint64_t full[kStages];       // TMA bytes of a stage landed
  uint64_t wready[kStages];     // dequantized weight tile written (8 warp arrivals)
  uint64_t empty[kStages];      // the MMAs that read a stage finished
  uint64_t cfull[kCodeSlots];
  uint64_t cempty[kCodeSlots];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;               // after an abort
  uint32_t tmem_base;
  uint32_t abort_flag;
  GroupTable groups;
};

constexpr size_t gemm_smem(bool i8) {
  return size_t(kStages) * kStageBytes + (i8 ? 0 : size_t(kCodeSlots) * kCodeBytes) + sizeof(GemmShared) + 1024;
}
static_assert(gemm_smem(false) <= 232448, "shared memory of one CTA");

// int8 x int8 -> int32 MMA and its instruction descriptor (kind::i8: D s32,
// A and B signed 8-bit, both K-major).
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void tma_load_stack(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  tma_load_3d(dst, map, bar, x, y, z);
}

struct Tile {
  int e;        // expert
  int t0, cnt;  // first token row, tokens
  int nt;       // tokens rounded up to 16
  int n0;       // first output
};

// Tile `id` of the list ordered by expert, then output tile, then token tile
// (the CTAs that run together share an expert's weight tiles and tokens).
// The tokens of an expert are cut into ceil(c / 256) tiles of one size.
__device__ __forceinline__ Tile tile_at(const GroupTable* g, int E, int col_tiles, int id) {
  Tile t;
  t.e = expert_of_tile(g, E, id / col_tiles);
  const int q = id - g->tiles[t.e] * col_tiles;
  const int parts = g->tiles[t.e + 1] - g->tiles[t.e];
  const int ct = q / parts, rt = q - ct * parts;
  const int first = g->start[t.e], end = g->start[t.e + 1];
  const int size = ((end - first + parts - 1) / parts + 15) & ~15;
  t.t0 = first + rt * size;
  t.cnt = min(size, end - t.t0);
  t.nt = (t.cnt + 15) & ~15;
  t.n0 = ct * kTileW;
  return t;
}

// Byte offset in a code box (128 rows of 64 bytes, 64-byte swizzle) of the 16
// code bytes that (row, half) of the weight tile needs at step j of the box.
// kFwd: box row = W row; kDx: box row = reduction index j * 64 + (row & 63),
// and the tile's k range takes two 32-byte column groups.
template <int MODE>
__device__ __forceinline__ uint32_t box_offset(uint32_t row, uint32_t half, uint32_t j) {
  const uint32_t R = MODE == kFwd ? row : j * 64u + (row & 63u);
  const uint32_t c = (MODE == kFwd ? 2u * j : 2u * (row >> 6)) + half;
  return R * 64u + ((c ^ ((R >> 1) & 3u)) << 4);
}

template <int MODE, bool F16>
__global__ void __launch_bounds__(MODE == kI8 ? 256 : 512, 1)
    expert_gemm_kernel(const __grid_constant__ ExpertMaps maps, const ExpertParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* code_base = smem + kStages * kStageBytes;
  GemmShared* sh = reinterpret_cast<GemmShared*>(code_base + (MODE == kI8 ? 0 : kCodeSlots * kCodeBytes));
  auto stage_w = [&](int s) { return smem + s * kStageBytes; };
  auto stage_t = [&](int s) { return smem + s * kStageBytes + kWBytes; };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sh->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh->full[s], MODE == kI8 ? 3 : 2);
      mbar_init(&sh->wready[s], kDeqWarps);
      mbar_init(&sh->empty[s], 1);
    }
    for (int c = 0; c < kCodeSlots; ++c) {
      mbar_init(&sh->cfull[c], 1);
      mbar_init(&sh->cempty[c], kDeqWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], 4);
    }
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch(&maps.tok_l);
    tma_prefetch(&maps.tok_s);
    tma_prefetch(&maps.w);
  }
  if (warp == 2) {
    if (p.offsets != nullptr) {
      build_groups(&sh->groups, p.offsets, p.E, p.M, kTileT, blockIdx.x == 0 ? p.status : nullptr);
    } else if (lane == 0) {
      sh->groups.start[0] = sh->groups.tiles[0] = 0;
      sh->groups.start[1] = p.M;
      sh->groups.tiles[1] = (p.M + kTileT - 1) / kTileT;
    }
  }
  if (warp == 3) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int tiles = sh->groups.tiles[p.E] * p.col_tiles;
  const int steps = p.main_steps + p.adapter_steps;

  if (warp < 2) {
    // ---------------- token producers: warp p loads rows 128 p .. of a tile in
    // 128-row boxes (32 p .. in 32-row boxes for up to 64 tokens)
    if (lane == 0) {
      if (MODE == kI8) grid_dep_wait();
      bool waited = false;
      int it = 0;
      bool ok = true;
      for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
        const Tile t = tile_at(&sh->groups, p.E, p.col_tiles, id);
        const bool large = t.nt > 64;
        const int rows = large ? 128 : 32;
        const bool loads = warp * rows < t.nt;
        const uint32_t bytes = loads ? uint32_t(rows) * 128u : 0u;
        const uint32_t at = uint32_t(warp * rows) * 128u;
        const CUtensorMap* tok = large ? &maps.tok_l : &maps.tok_s;
        const CUtensorMap* ad = large ? &maps.ad_l : &maps.ad_s;
        for (int k = 0; k < steps; ++k, ++it) {
          const int s = it % kStages;
          ok = mbar_wait(&sh->empty[s], ((it / kStages) & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          if (k < p.main_steps) {
            mbar_arrive_expect_tx(&sh->full[s], bytes);
            if (loads) tma_load_2d(stage_t(s) + at, tok, &sh->full[s], k * (MODE == kI8 ? 128 : 64), t.t0 + warp * rows);
          } else {
            if (!waited) grid_dep_wait();     // T or U: the kernel before
            waited = true;
            const int r0 = (k - p.main_steps) * 64;
            mbar_arrive_expect_tx(&sh->full[s], bytes + (warp == 0 ? kWBytes : 0u));
            if (loads) tma_load_2d(stage_t(s) + at, ad, &sh->full[s], r0, t.t0 + warp * rows);
            if (warp == 0) {
              if (MODE == kFwd) {
                tma_load_stack(stage_w(s), &maps.wad, &sh->full[s], r0, t.n0, t.e);
              } else {
                tma_load_stack(stage_w(s), &maps.wad, &sh->full[s], t.n0, r0, t.e);
                tma_load_stack(stage_w(s) + 8192, &maps.wad, &sh->full[s], t.n0 + 64, r0, t.e);
              }
            }
          }
        }
      }
      if (*abort_flag)   // unwind: wait (bounded) for the copies in flight
        for (int j = std::max(0, it - kStages); j < it; ++j) {
          uint32_t none = 0;
          mbar_wait(&sh->full[j % kStages], (j / kStages) & 1, &none, nullptr);
        }
    }
  } else if (warp == 2) {
    // ---------------- weight-side producer
    if (lane == 0) {
      if (MODE == kI8) grid_dep_wait();
      int it = 0;
      bool ok = true;
      const int groups = MODE == kI8 ? p.main_steps : (p.main_steps + kCodeSteps - 1) / kCodeSteps;
      for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
        const Tile t = tile_at(&sh->groups, p.E, p.col_tiles, id);
        for (int g = 0; g < groups; ++g, ++it) {
          if (MODE == kI8) {
            const int s = it % kStages;
            ok = mbar_wait(&sh->empty[s], ((it / kStages) & 1) ^ 1, abort_flag, p.status);
            if (!ok) break;
            mbar_arrive_expect_tx(&sh->full[s], kWBytes);
            tma_load_stack(stage_w(s), &maps.w, &sh->full[s], g * 128, t.n0, t.e);
          } else {
            const int c = it % kCodeSlots;
            ok = mbar_wait(&sh->cempty[c], ((it / kCodeSlots) & 1) ^ 1, abort_flag, p.status);
            if (!ok) break;
            mbar_arrive_expect_tx(&sh->cfull[c], kCodeBytes);
            uint8_t* dst = code_base + c * kCodeBytes;
            if (MODE == kFwd) tma_load_stack(dst, &maps.w, &sh->cfull[c], g * 64, t.n0, t.e);
            else tma_load_stack(dst, &maps.w, &sh->cfull[c], t.n0 / 2, g * 128, t.e);
          }
        }
      }
      if (*abort_flag) {
        const int ring = MODE == kI8 ? kStages : kCodeSlots;
        for (int j = std::max(0, it - ring); j < it; ++j) {
          uint32_t none = 0;
          mbar_wait(MODE == kI8 ? &sh->full[j % ring] : &sh->cfull[j % ring], (j / ring) & 1, &none, nullptr);
        }
      }
    }
  } else if (warp == 3) {
    // ---------------- MMA issuer
    if (lane == 0) {
      int it = 0, n = 0;
      bool ok = true;
      for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x, ++n) {
        const Tile t = tile_at(&sh->groups, p.E, p.col_tiles, id);
        const uint32_t idesc = MODE == kI8 ? idesc_i8(128, t.nt) : idesc_f32acc(128, t.nt, MODE == kDx, false, F16);
        const uint32_t d = tmem + uint32_t(n & 1) * 256u;
        ok = mbar_wait(&sh->acc_empty[n & 1], ((n >> 1) & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        for (int k = 0; k < steps; ++k, ++it) {
          const int s = it % kStages;
          const uint32_t ph = (it / kStages) & 1;
          ok = mbar_wait(&sh->full[s], ph, abort_flag, p.status);
          if (ok && MODE != kI8) ok = mbar_wait(&sh->wready[s], ph, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t w_base = smem_u32(stage_w(s));
          const uint32_t t_base = smem_u32(stage_t(s));
          int ksub = 4;
          if (MODE != kI8 && k >= p.main_steps) {
            const int left = p.r - (k - p.main_steps) * 64;
            ksub = left >= 64 ? 4 : (left + 15) / 16;
          }
          for (int kk = 0; kk < ksub; ++kk) {
            const uint64_t adesc = MODE == kDx ? smem_desc_sw128(w_base + kk * 2048, 8192, 1024)
                                               : smem_desc_sw128(w_base + kk * 32, 16, 1024);
            const uint64_t bdesc = smem_desc_sw128(t_base + kk * 32, 16, 1024);
            const uint32_t acc = (k > 0 || kk > 0) ? 1u : 0u;
            if (MODE == kI8) umma_i8(d, adesc, bdesc, idesc, acc);
            else umma_f16(d, adesc, bdesc, idesc, acc);
          }
          umma_commit(&sh->empty[s]);
        }
        if (ok) umma_commit(&sh->acc_full[n & 1]);
      }
      if (!ok) {   // unwind: wait (bounded) for the MMAs in flight
        umma_commit(&sh->drain);
        uint32_t none = 0;
        mbar_wait(&sh->drain, 0, &none, nullptr);
      }
    }
  } else if (warp < kDeqWarp) {
    // ---------------- epilogue: lane = output n, register = token
    if (MODE == kI8) grid_dep_wait();
    const int quad = warp - kEpiWarp;
    int n = 0;
    for (int id = blockIdx.x; id < tiles; id += gridDim.x, ++n) {
      const Tile t = tile_at(&sh->groups, p.E, p.col_tiles, id);
      const int col = t.n0 + quad * 32 + lane;
      const bool col_ok = col < p.out_cols;
      float bias = 0.0f, sw = 0.0f;
      if (col_ok) {
        const int64_t at = int64_t(t.e) * p.out_cols + col;
        if (MODE == kI8) sw = __ldg(p.w_scale + at);
        if (p.bias != nullptr) {
          if (MODE == kI8 && p.out_dtype == NF4_F32) bias = __ldg(static_cast<const float*>(p.bias) + at);
          else if (MODE == kI8 ? p.out_dtype == NF4_F16 : F16) bias = __half2float(static_cast<const __half*>(p.bias)[at]);
          else bias = __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[at]);
        }
      }
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&sh->acc_full[n & 1], (n >> 1) & 1, abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c * 32 < t.cnt; ++c) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + uint32_t(n & 1) * 256u + c * 32, v);
        float sx = 0.0f;
        if (MODE == kI8 && c * 32 + lane < t.cnt) sx = __ldg(p.x_scale + t.t0 + c * 32 + lane);
        tmem_ld_wait();
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (MODE == kI8)
            f[i] = __fmul_rn(__fmul_rn(float(int(v[i])), __shfl_sync(0xffffffffu, sx, i)), sw);
          else
            f[i] = __uint_as_float(v[i]);
          if (p.bias != nullptr) f[i] = __fadd_rn(f[i], bias);
        }
        const int left = t.cnt - c * 32;
        const int64_t row0 = int64_t(t.t0) + c * 32;
        if (MODE == kI8 && p.out_dtype == NF4_F32) {
          float* o = static_cast<float*>(p.out) + row0 * p.out_cols + col;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (col_ok && i < left) o[int64_t(i) * p.out_cols] = f[i];
        } else {
          // two lanes trade so that each stores two neighbouring outputs of one token
          const bool odd = lane & 1;
          const bool f16 = MODE == kI8 ? p.out_dtype == NF4_F16 : F16;
          uint16_t* o = static_cast<uint16_t*>(p.out) + (row0 + odd) * p.out_cols + (col & ~1);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? f[i] : f[i + 1], 1);
            const uint32_t two = pack2(f16, odd ? got : f[i], odd ? f[i + 1] : got);
            if (col_ok && i + int(odd) < left) *reinterpret_cast<uint32_t*>(o + int64_t(i) * p.out_cols) = two;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->acc_empty[n & 1]);
    }
  } else {
    // ---------------- dequant warps: two threads per weight-tile row (16 rows a
    // warp), half an NF4 chunk of 64 each
    const int row = (warp - kDeqWarp) * 16 + (lane & 15);
    const uint32_t half = uint32_t(lane >> 4);
    const bool dq = p.dq != 0;
    const float s_g = dq ? __ldg(p.absmax_scale) : 0.0f;
    int it = 0, box = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
      const Tile t = tile_at(&sh->groups, p.E, p.col_tiles, id);
      const int64_t first = int64_t(t.e) * p.w_rows;
      auto scale_at = [&](int k) -> float {
        if (k >= p.main_steps) return 0.0f;
        const int wr = MODE == kFwd ? t.n0 + row : k * 64 + (row & 63);
        const int ch = MODE == kFwd ? k : (t.n0 >> 6) + (row >> 6);
        if (wr >= p.w_rows || ch * 64 >= p.w_cols) return 0.0f;   // zero rows: the codes there are 0 too
        return load_scale(p.absmax_q, p.absmax, s_g, dq, chunk_block(first + wr, p.w_cols, ch, p.bs_shift));
      };
      float sc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[j] = scale_at(j);
      for (int k = 0; k < steps; ++k, ++it) {
        const int s = it % kStages;
        const float scale = sc[0];
        sc[0] = sc[1];
        sc[1] = sc[2];
        sc[2] = sc[3];
        sc[3] = scale_at(k + 4);
        bool good = mbar_wait(&sh->empty[s], ((it / kStages) & 1) ^ 1, abort_flag, p.status);
        const bool main = k < p.main_steps;
        const int j = k % kCodeSteps;
        if (good && main && j == 0)
          good = mbar_wait(&sh->cfull[box % kCodeSlots], (box / kCodeSlots) & 1, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, good);
        if (!ok) break;
        if (main) {
          dequant_half_row(code_base + (box % kCodeSlots) * kCodeBytes + box_offset<MODE>(uint32_t(row), half, uint32_t(j)),
                           scale, stage_w(s), uint32_t(row), half, F16);
          fence_proxy_async_smem();
        }
        __syncwarp();
        // one arrival per step, adapter steps too, so the phases of wready follow the ring
        if (lane == 0) mbar_arrive(&sh->wready[s]);
        if (main && (j == kCodeSteps - 1 || k == p.main_steps - 1)) {
          if (lane == 0) mbar_arrive(&sh->cempty[box % kCodeSlots]);
          ++box;
        }
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

// ------------------------------------------------------------------ host side

PerDeviceOnce g_attr_done;

cudaError_t set_attrs() {
  const int dev = PerDeviceOnce::current();
  if (g_attr_done.done(dev)) return cudaSuccess;
  const void* nf4[4] = {(const void*)expert_gemm_kernel<kFwd, false>, (const void*)expert_gemm_kernel<kFwd, true>,
                        (const void*)expert_gemm_kernel<kDx, false>, (const void*)expert_gemm_kernel<kDx, true>};
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i)
    e = cudaFuncSetAttribute(nf4[i], cudaFuncAttributeMaxDynamicSharedMemorySize, int(gemm_smem(false)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute((const void*)expert_gemm_kernel<kI8, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(gemm_smem(true)));
  if (e == cudaSuccess) g_attr_done.mark(dev);
  return e;
}

bool set_grid(ExpertGemm* L, int sms) {
  ExpertParams& p = L->p;
  p.col_tiles = int((int64_t(p.out_cols) + kTileW - 1) / kTileW);
  const int64_t tiles = max_row_tiles(p.M, p.E, kTileT) * p.col_tiles;
  if (tiles > int64_t(0x7fffffff)) return false;
  L->grid = unsigned(std::min<int64_t>(tiles, sms));
  return true;
}

// Tokens [M, cols] and the adapter activation [M, r], in both box heights.
bool token_maps(ExpertGemm* L, const void* tok, uint64_t cols, const void* ad, int r, uint64_t M) {
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  return encode_map_2d(&L->maps.tok_l, tok, MapElem::k16, cols, M, 64, 128, sw) &&
         encode_map_2d(&L->maps.tok_s, tok, MapElem::k16, cols, M, 64, 32, sw) &&
         encode_map_2d(&L->maps.ad_l, ad, MapElem::k16, r, M, 64, 128, sw) &&
         encode_map_2d(&L->maps.ad_s, ad, MapElem::k16, r, M, 64, 32, sw);
}

template <int MODE, bool F16>
cudaError_t launch(const ExpertGemm& L, int prof_id, cudaStream_t st, int* launches) {
  cudaError_t e = set_attrs();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L.grid, 1, 1);
  cfg.blockDim = dim3(MODE == kI8 ? 256 : 512, 1, 1);
  cfg.dynamicSmemBytes = gemm_smem(MODE == kI8);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = prof_on() ? 0 : 1;
  NF4_PROF_BEGIN(st, prof_id);
  e = cudaLaunchKernelEx(&cfg, expert_gemm_kernel<MODE, F16>, L.maps, L.p);
  NF4_PROF_END(st, prof_id);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace

bool ExpertGemm::prepare(const GroupedArgs& g, bool backward, const void* ad, int sms) {
  const LinearArgs& a = g.lin;
  dx = backward;
  f16 = a.f16 != 0;
  ExpertGemm* L = this;
  const uint64_t N = uint64_t(a.N), K = uint64_t(a.K), E = uint64_t(g.E);
  const CUtensorMapSwizzle s128 = CU_TENSOR_MAP_SWIZZLE_128B, s64 = CU_TENSOR_MAP_SWIZZLE_64B;
  bool ok = token_maps(L, backward ? a.dy : a.x, backward ? N : K, ad, a.r, uint64_t(a.M));
  // code boxes: 128 W rows x 64 bytes (kFwd: two K steps of a row tile; kDx: two
  // reduction steps of 128 columns)
  ok = ok && encode_map_stack(&L->maps.w, a.w->codes, MapElem::kU8, K / 2, N, E, 64, 128, s64);
  ok = ok && (backward ? encode_map_stack(&L->maps.wad, a.A, MapElem::k16, K, uint64_t(a.r), E, 64, 64, s128)
                       : encode_map_stack(&L->maps.wad, a.B, MapElem::k16, uint64_t(a.r), N, E, 64, 128, s128));
  p = ExpertParams{};
  p.M = int(a.M);
  p.E = g.E;
  p.out_cols = int(backward ? a.K : a.N);
  p.w_rows = int(a.N);
  p.w_cols = int(a.K);
  p.r = a.r;
  p.main_steps = int(backward ? (a.N + 63) / 64 : a.K / 64);
  p.adapter_steps = (a.r + 63) / 64;
  p.bs_shift = log2_block(a.w->block_size);
  p.dq = a.w->double_quant;
  p.offsets = g.offsets;
  p.absmax_q = a.w->absmax_q;
  p.absmax = a.w->absmax;
  p.absmax_scale = a.w->absmax_scale;
  p.bias = backward ? nullptr : a.bias;
  p.out = backward ? a.dx : a.y;
  p.status = a.status;
  return ok && set_grid(L, sms);
}

cudaError_t ExpertGemm::run(cudaStream_t st, int* launches) const {
  if (dx) return f16 ? launch<kDx, true>(*this, kKGroupedDx, st, launches) : launch<kDx, false>(*this, kKGroupedDx, st, launches);
  return f16 ? launch<kFwd, true>(*this, kKGroupedFwd, st, launches) : launch<kFwd, false>(*this, kKGroupedFwd, st, launches);
}

cudaError_t launch_int8_gemm(const Int8LinearArgs& a, int sms, cudaStream_t st, int* launches) {
  ExpertGemm L;
  const CUtensorMapSwizzle s128 = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t M = uint64_t(a.M), N = uint64_t(a.N), K = uint64_t(a.K);
  bool ok = encode_map_2d(&L.maps.tok_l, a.x, MapElem::kU8, K, M, 128, 128, s128) &&
            encode_map_2d(&L.maps.tok_s, a.x, MapElem::kU8, K, M, 128, 32, s128) &&
            encode_map_stack(&L.maps.w, a.w, MapElem::kU8, K, N, 1, 128, 128, s128);
  L.maps.ad_l = L.maps.ad_s = L.maps.wad = L.maps.w;   // not used
  ExpertParams& p = L.p;
  p = ExpertParams{};
  p.M = int(a.M);
  p.E = 1;
  p.out_cols = p.w_rows = int(a.N);
  p.w_cols = int(a.K);
  p.main_steps = int((a.K + 127) / 128);
  p.out_dtype = a.dtype;
  p.bias = a.bias;
  p.out = a.y;
  p.w_scale = a.w_scale;
  p.x_scale = a.x_scale;
  p.status = a.status;
  if (!ok || !set_grid(&L, sms)) return cudaErrorInvalidValue;
  return launch<kI8, false>(L, kKInt8Linear, st, launches);
}

}  // namespace nf4
