// The big products of the expert layer and of the 8-bit linear on the sm_100a
// tensor cores, rows sorted by expert:
//   kFwd   y[m, n]  = sum_k W'_e[n, k] x[m, k] + sum_j B_e[n, j] T[m, j] (+ bias_e[n])
//   kDx    dx[m, k] = sum_n W'_e[n, k] dy[m, n] + sum_j A_e[j, k] U[m, j]
//   kI8    y[m, n]  = (sum_k wq[n, k] xq[m, k]) sx[m] sw[n] (+ bias[n])
//
// The weight is the A operand of the MMA (an expert's outputs on the TMEM
// lanes) and the tokens are the B operand, whose count is any multiple of 16 up
// to 256: an expert's ragged rows are cut into even tiles that waste at most 15
// columns, where tokens on the lanes would waste up to 127.  A tile has one or
// two such MMAs (parts): the second takes the same decoded weight tile, so that
// a weight is decoded once for 512 tokens.  The layout also puts the
// outputs' contiguous dimension on the lanes, so a row's results are stored
// under its own row predicate and rows of other experts stay untouched.
//
// Two CTAs on two SMs form a pair (cta_group::2, M = 256): each holds 128 of a
// tile's 256 weight rows and half of its tokens, so the tokens' shared-memory
// traffic, which bounds a single CTA (104 KB a step of 512 MMA cycles at 128
// bytes a cycle), is shared.  Persistent pairs walk over (expert, 256 outputs,
// token tile); the tile list comes from the offsets in device memory, scanned
// once per CTA.
// Roles in each CTA: warp 0 token TMA, warp 1 weight-side TMA (NF4 codes or the
// int8 tile), warp 2 MMA (issued by the pair's leader), warps 4-7 epilogue,
// warps 8-19 dequant (NF4).  Rings: six stages of [weight tile 16 KB | tokens
// 16 KB], or four with 32 KB of tokens; six code slots; two accumulators of 256
// TMEM columns, so that a one-part tile's epilogue runs under the next tile's
// MMAs, and a two-part tile's first half under the next tile's first steps.
//
// What bounds it.  One part: the decode (a step of 64 has 512 cycles of MMAs and
// about 930 of decoding), so the time hardly depends on the rows.  Two parts: the
// tensor pipe is active for 65 % of the time (4096 x 4096, 4096 rows of 4 experts,
// 155 us), with MMA operands, TMA writes and decoded tiles on the same
// shared-memory port; back to back the power limit.  y of 8192 rows on 8 experts of
// 11008 x 4096 (739 GFLOP): 594 us alone, 690 us back to back.  kI8, 4096 x 11008 x
// 4096: 112 us, tensor pipe 90 % active.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "expert_gemm.h"
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
using namespace expert;

constexpr int kFwd = 0;
constexpr int kDx = 1;
constexpr int kI8 = 2;

constexpr int kTileW = 256;                 // outputs per tile, 128 in each CTA
constexpr int kPartT = 256;                 // tokens of one MMA at most, half in each CTA
constexpr uint32_t kWBytes = 128 * 128;     // weight tile of a CTA: 128 x 128 bytes
constexpr uint32_t kTBytes = 128 * 128;     // its tokens of one part
constexpr uint32_t kCodeBytes = 128 * 32;   // kDx: NF4 codes of one step
constexpr int kCodeSlots = 6;
constexpr int kEpiWarp = 4;                 // warps 4..7
constexpr int kDeqWarp = 8;

// Ring stages: [weight tile | tokens of each part].
constexpr int stages_of(int parts) { return parts == 2 ? 4 : 6; }
// Dequant groups of four warps each take every deq_groups-th step; the stages and
// the code slots are multiples of their number, so that each belongs to one group.
constexpr int deq_groups(int parts) { return parts == 2 ? 2 : 3; }
constexpr int threads_of(int mode, int parts) { return 32 * (kDeqWarp + (mode == kI8 ? 0 : 4 * deq_groups(parts))); }
constexpr uint32_t stage_bytes_of(int parts) { return kWBytes + uint32_t(parts) * kTBytes; }

struct GemmShared {
  uint64_t full[stages_of(1)];  // leader: both CTAs' bytes landed and weight tiles written
  uint64_t empty[stages_of(1)]; // the MMAs that read a stage finished
  uint64_t cfull[kCodeSlots];   // kDx: a step's codes landed
  uint64_t cempty[kCodeSlots];  // kDx: and were read
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;               // after an abort
  uint32_t tmem_base;
  uint32_t abort_flag;
  GroupTable groups;
};

constexpr size_t gemm_smem(int mode, int parts) {
  return size_t(stages_of(parts)) * stage_bytes_of(parts) + (mode == kDx ? kCodeSlots * kCodeBytes : 0) +
         sizeof(GemmShared) + 1024;
}
static_assert(gemm_smem(kDx, 1) <= 232448 && gemm_smem(kDx, 2) <= 232448, "shared memory of one CTA");

// int8 x int8 -> int32 MMA and its instruction descriptor (kind::i8: D s32,
// A and B signed 8-bit, both K-major).
__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// 3-D tiled load into this CTA whose bytes complete on the leader's barrier.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster_addr,
                                                 int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Arrive on a barrier of the pair's leader, releasing at cluster scope: the waiter
// may be in the other CTA.  What the arrival announces are operand tiles in this
// CTA's shared memory, which fence.proxy.async has handed to the async proxy, or
// accumulators whose reads tcgen05.wait has completed.  So the release is restricted
// to this CTA's shared memory; a full one waits for every store in flight, the
// epilogue's output included (y of 8192 rows on 8 experts of 11008 x 4096: 894 us
// against 715).
__device__ __forceinline__ void arrive_leader(uint32_t cluster_addr) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
      : "memory");
}

struct Tile {
  int e;        // expert
  int t0, cnt;  // first token row, tokens
  int nt[2];    // MMA columns of the parts (multiples of 16; 0: no second part)
  int n0;       // first output
};

// Tile `id` of the list ordered by expert, then output tile, then token tile
// (the pairs that run together share an expert's weight tiles and tokens).
// The tokens of an expert are cut into ceil(c / (256 PARTS)) tiles of one size.
template <int PARTS>
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
  const int nt = (t.cnt + 15) & ~15;
  t.nt[0] = PARTS == 2 && nt > kPartT ? ((nt >> 1) + 15) & ~15 : nt;
  t.nt[1] = nt - t.nt[0];
  t.n0 = ct * kTileW;
  return t;
}

// Byte offset in a step's code slot (kDx: 64 reduction rows of 64 bytes, the
// tile's k range, 64-byte swizzle) of the first of the two 16-byte chunks that
// weight-tile row `row` needs: k group row >> 6 of reduction row row & 63.  The
// second is at that offset ^ 16.  Eight consecutive rows read from eight
// different bank groups.
__device__ __forceinline__ uint32_t code_offset(uint32_t row) {
  const uint32_t R = row & 63u, c = 2u * (row >> 6);
  return R * 64u + ((c ^ ((R >> 1) & 3u)) << 4);
}

template <int MODE, bool F16, int PARTS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(MODE, PARTS), 1)
    expert_gemm_kernel(const __grid_constant__ ExpertMaps maps, const ExpertParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = expert::align_1024(smem_raw);
  constexpr int kStages = stages_of(PARTS);
  constexpr int kDeqGroups = deq_groups(PARTS);
  static_assert(kStages % kDeqGroups == 0 && kCodeSlots % kDeqGroups == 0, "a stage and a slot belong to one group");
  constexpr uint32_t kStageBytes = stage_bytes_of(PARTS);
  uint8_t* code_base = smem + kStages * kStageBytes;
  GemmShared* sh = reinterpret_cast<GemmShared*>(code_base + (MODE == kDx ? kCodeSlots * kCodeBytes : 0));
  auto stage_w = [&](int s) { return smem + s * kStageBytes; };
  auto stage_t = [&](int s) { return smem + s * kStageBytes + kWBytes; };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  volatile uint32_t* abort_flag = &sh->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      // leader: its token producer (which expects every byte) and the dequant
      // warps of both CTAs
      mbar_init(&sh->full[s], MODE == kI8 ? 1 : 1 + 8);
      mbar_init(&sh->empty[s], 1);
    }
    for (int s = 0; s < kCodeSlots; ++s) {
      mbar_init(&sh->cfull[s], 1);
      mbar_init(&sh->cempty[s], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], 8);   // leader: the epilogue warps of both CTAs
    }
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch(&maps.tok_l);
    tma_prefetch(&maps.tok_s);
    if (MODE != kFwd) tma_prefetch(&maps.w);
  }
  if (warp == 1) {
    if (p.offsets != nullptr) {
      build_groups(&sh->groups, p.offsets, p.E, p.M, PARTS * kPartT, blockIdx.x == 0 ? p.status : nullptr);
    } else if (lane == 0) {
      sh->groups.start[0] = sh->groups.tiles[0] = 0;
      sh->groups.start[1] = p.M;
      sh->groups.tiles[1] = (p.M + kPartT - 1) / kPartT;
    }
  }
  if (warp == 2) {
    tmem_alloc_pair(&sh->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int tiles = sh->groups.tiles[p.E] * p.col_tiles;
  const int steps = p.main_steps + p.adapter_steps;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto leader_bar = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };

  // The single-issuer roles run as whole warps with one elected lane, so that
  // their counters and addresses stay in uniform registers (issued from a
  // divergent lane, the four MMAs of a step took 770 cycles).
  if (warp == 0) {
    // ---------------- tokens: this CTA's half of the tile, in a 128-row box (or
    // a 32-row one)
    const bool issue = elect_one();
    if (MODE == kI8) grid_dep_wait();
    bool waited = false, ok = true;
    int s = 0, issued = 0;
    uint32_t ph = 1;
    for (int id = pair; id < tiles && ok; id += pairs) {
      const Tile t = tile_at<PARTS>(&sh->groups, p.E, p.col_tiles, id);
      const int half = t.nt[0] >> 1;
      const bool large = half > 32;
      const bool two = PARTS == 2 && t.nt[1] > 0;
      const uint32_t bytes = two ? 2 * kTBytes : large ? kTBytes : 32u * 128u;   // of one CTA
      const int y = t.t0 + int(rank) * half;
      const int y2 = t.t0 + t.nt[0] + int(rank) * (t.nt[1] >> 1);
      const CUtensorMap* tok = large ? &maps.tok_l : &maps.tok_s;
      const CUtensorMap* ad = large ? &maps.ad_l : &maps.ad_s;
      for (int k = 0; k < steps; ++k) {
        ok = ring_wait(&sh->empty[s], ph, abort_flag, p.status);
        if (!ok) break;
        const bool main = k < p.main_steps;
        if (!main && !waited) grid_dep_wait();     // T or U: the kernel before
        waited |= !main;
        if (issue) {
          const uint32_t bar = leader_bar(&sh->full[s]);
          if (rank == 0) mbar_arrive_expect_tx(&sh->full[s], 2 * (bytes + (MODE == kI8 || !main ? kWBytes : 0u)));
          if (main) {
            tma_load_2d_pair(stage_t(s), tok, bar, k * (MODE == kI8 ? 128 : 64), y);
            if (two) tma_load_2d_pair(stage_t(s) + kTBytes, tok, bar, k * 64, y2);
          } else {
            const int r0 = (k - p.main_steps) * 64, n0 = t.n0 + 128 * int(rank);
            tma_load_2d_pair(stage_t(s), ad, bar, r0, y);
            if (two) tma_load_2d_pair(stage_t(s) + kTBytes, ad, bar, r0, y2);
            if (MODE == kFwd) {
              tma_load_3d_pair(stage_w(s), &maps.wad, bar, r0, n0, t.e);
            } else {
              tma_load_3d_pair(stage_w(s), &maps.wad, bar, n0, r0, t.e);
              tma_load_3d_pair(stage_w(s) + 8192, &maps.wad, bar, n0 + 64, r0, t.e);
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
    }
    // Without a tile too: what runs after this grid may count on the kernel before it
    // being done (it may read the offsets still when no row belongs to an expert).
    if (MODE != kI8 && !waited) grid_dep_wait();
    if (*abort_flag)   // unwind: wait (bounded) for the stages in flight
      for (int j = max(0, issued - kStages); j < issued; ++j) {
        uint32_t none = 0;
        ring_wait(&sh->empty[j % kStages], (j / kStages) & 1, &none, nullptr);
      }
  } else if (warp == 1) {
    // ---------------- weight side: the int8 tile of every step (kI8), or the
    // codes of every main step (kDx)
    if (MODE != kFwd) {
      const bool issue = elect_one();
      if (MODE == kI8) grid_dep_wait();
      constexpr int kSlots = MODE == kI8 ? kStages : kCodeSlots;
      int s = 0;
      uint32_t ph = (1u << kSlots) - 1;   // bit s: parity of the wait for slot s, toggled at each use
      bool ok = true;
      for (int id = pair; id < tiles && ok; id += pairs) {
        const Tile t = tile_at<PARTS>(&sh->groups, p.E, p.col_tiles, id);
        const int n0 = t.n0 + 128 * int(rank);
        for (int k = 0; k < steps; ++k) {
          if (k < p.main_steps) {
            ok = ring_wait(MODE == kI8 ? &sh->empty[s] : &sh->cempty[s], (ph >> s) & 1u, abort_flag, p.status);
            if (!ok) break;
            ph ^= 1u << s;
            if (issue) {
              if (MODE == kI8) {
                tma_load_3d_pair(stage_w(s), &maps.w, leader_bar(&sh->full[s]), k * 128, n0, t.e);
              } else {
                mbar_arrive_expect_tx(&sh->cfull[s], kCodeBytes);
                tma_load_3d(code_base + s * kCodeBytes, &maps.w, &sh->cfull[s], n0 / 2, k * 64, t.e);
              }
            }
            __syncwarp();
          }
          if (++s == kSlots) s = 0;
        }
      }
      if (MODE == kDx && *abort_flag)   // unwind: wait (bounded) for the codes in flight
        for (int j = 0; j < kCodeSlots; ++j) {
          uint32_t none = 0;
          ring_wait(&sh->cfull[j], (ph >> j) & 1u, &none, nullptr);
        }
    }
  } else if (warp == 2) {
    // ---------------- MMA: the leader's warp walks the steps, one lane issues
    if (rank == 0) {
      const bool issue = elect_one();
      // descriptors of stage 0; a stage is kStageBytes further, a K substep 32
      // bytes (K-major) or 16 rows of 128 bytes (MN-major)
      const uint64_t w_desc = MODE == kDx ? smem_desc_sw128(smem_u32(stage_w(0)), 8192, 1024)
                                          : smem_desc_sw128(smem_u32(stage_w(0)), 16, 1024);
      const uint64_t t_desc = smem_desc_sw128(smem_u32(stage_t(0)), 16, 1024);
      constexpr uint32_t kWSub = (MODE == kDx ? 2048 : 32) >> 4, kTSub = 32 >> 4;
      int s = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int id = pair; id < tiles && ok; id += pairs) {
        const Tile t = tile_at<PARTS>(&sh->groups, p.E, p.col_tiles, id);
        const int parts = PARTS == 2 && t.nt[1] > 0 ? 2 : 1;
        for (int k = 0; k < steps && ok; ++k) {
          ok = mbar_wait_cluster(&sh->full[s], ph, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t wd = w_desc + uint32_t(s) * (kStageBytes >> 4);
          const int left = MODE == kI8 || k < p.main_steps ? 64 : p.r - (k - p.main_steps) * 64;
#pragma unroll
          for (int h = 0; h < PARTS; ++h) {
            if (h >= parts) break;
            const int b = (n + h) & 1;
            if (k == 0) {
              ok = mbar_wait_cluster(&sh->acc_empty[b], (((n + h) >> 1) & 1) ^ 1, abort_flag, p.status);
              if (!ok) break;
              tc_fence_after();
            }
            const uint32_t d = tmem + uint32_t(b) * 256u;
            const uint32_t idesc = MODE == kI8 ? idesc_i8(256, t.nt[h]) : idesc_f32acc(256, t.nt[h], MODE == kDx, false, F16);
            const uint64_t td = t_desc + uint32_t(s) * (kStageBytes >> 4) + uint32_t(h) * (kTBytes >> 4);
            if (issue) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint32_t acc = (k > 0 || kk > 0) ? 1u : 0u;
                if (MODE == kI8) umma_i8_pair(d, wd + kk * kWSub, td + kk * kTSub, idesc, acc);
                else if (kk * 16 < left) umma_f16_pair(d, wd + kk * kWSub, td + kk * kTSub, idesc, acc);
              }
              // The last step's commits go to the accumulators' barriers; the
              // epilogue then releases that step's stage.  MMAs finish in order,
              // so a commit covers the whole accumulation.
              if (k + 1 == steps) umma_commit_pair_mc(&sh->acc_full[b], 0x3);
              else if (h + 1 == parts) umma_commit_pair_mc(&sh->empty[s], 0x3);
            }
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        n += parts;
      }
      if (!ok && issue) {   // unwind: wait (bounded) for the MMAs in flight
        umma_commit_pair_mc(&sh->drain, 0x1);
        uint32_t none = 0;
        ring_wait(&sh->drain, 0, &none, nullptr);
      }
    }
  } else if (warp >= kEpiWarp && warp < kDeqWarp) {
    // ---------------- epilogue: lane = output n, register = token
    if (MODE == kI8) grid_dep_wait();
    const int quad = warp - kEpiWarp;
    int n = 0, last = 0;   // last: stage of the tile's last step
    bool ok = true;
    for (int id = pair; id < tiles && ok; id += pairs) {
      const Tile t = tile_at<PARTS>(&sh->groups, p.E, p.col_tiles, id);
      const int col = t.n0 + 128 * int(rank) + quad * 32 + lane;
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
      last = (last + steps) % kStages;
      const int parts = PARTS == 2 && t.nt[1] > 0 ? 2 : 1;
#pragma unroll 1
      for (int h = 0; h < PARTS; ++h, ++n) {
        if (h >= parts) break;
        const int t0 = h == 0 ? t.t0 : t.t0 + t.nt[0];
        const int cnt = h + 1 == parts ? t.t0 + t.cnt - t0 : t.nt[0];
        ok = warp_wait<300>(&sh->acc_full[n & 1], (n >> 1) & 1, abort_flag, p.status);
        if (!ok) break;
        if (h + 1 == parts && quad == 0 && lane == 0) mbar_arrive(&sh->empty[(last + kStages - 1) % kStages]);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c * 32 < cnt; ++c) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + uint32_t(n & 1) * 256u + c * 32, v);
          float sx = 0.0f;
          if (MODE == kI8 && c * 32 + lane < cnt) sx = __ldg(p.x_scale + t0 + c * 32 + lane);
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
          const int left = cnt - c * 32;
          const int64_t row0 = int64_t(t0) + c * 32;
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
        if (lane == 0) arrive_leader(leader_bar(&sh->acc_empty[n & 1]));
      }
    }
  } else if (warp >= kDeqWarp) {
    // ---------------- dequant warps: one thread per weight-tile row and step, so
    // the table of a block's sixteen values is built once.  A group of four warps
    // takes every kDeqGroups-th step: decoding (codes to registers) needs no free
    // stage, so it runs ahead of the MMAs, and only the stores wait for the stage.
    const int group = (warp - kDeqWarp) >> 2;
    const int row = threadIdx.x & 127;
    const bool dq = p.dq != 0;
    const float s_g = dq ? __ldg(p.absmax_scale) : 0.0f;
    int base = 0;         // steps of the tiles before
    int s = group;               // stage of this group's next step
    uint32_t ph = 1;             // parity of the wait for that stage
    int own_slot = group;        // and its code slot (with as many stages as slots: the stage's)
    uint32_t cph = 0;            // bit i: parity of the wait for the codes in slot i
    bool ok = true;
    for (int id = pair; id < tiles && ok; id += pairs) {
      const Tile t = tile_at<PARTS>(&sh->groups, p.E, p.col_tiles, id);
      // this row's 64-element chunk at step k: c0 + k * c_step, counted over the
      // whole stack; its scale is that of the block that holds it
      const int n0 = t.n0 + 128 * int(rank);
      const int wr0 = MODE == kFwd ? n0 + row : row & 63;
      const int ch0 = MODE == kFwd ? 0 : (n0 >> 6) + (row >> 6);
      const uint32_t per_row = uint32_t(p.w_cols) >> 6;
      const uint32_t c0 = (uint32_t(t.e) * uint32_t(p.w_rows) + uint32_t(wr0)) * per_row + uint32_t(ch0);
      const uint32_t c_step = MODE == kFwd ? 1u : 64u * per_row;
      // rows past the expert's weight decode to zeros: their scale counts as 0 (and
      // their loads read the last row that is there, or the expert's first)
      const int k_end = MODE == kFwd ? (wr0 < p.w_rows ? p.main_steps : 0)
                                     : (uint32_t(ch0) < per_row ? (p.w_rows - wr0 + 63) >> 6 : 0);
      const uint32_t c_base = k_end > 0 ? c0 : uint32_t(t.e) * uint32_t(p.w_rows) * per_row;
      auto chunk_at = [&](int k) { return c_base + uint32_t(max(min(k, k_end - 1), 0)) * c_step; };
      // Scales are loaded two of this thread's steps ahead and converted only
      // where they are used, so that no step waits for a load.
      auto raw_scale = [&](int k) -> uint32_t {
        const uint32_t b = chunk_at(k) >> p.block_chunks_shift;
        return dq ? uint32_t(__ldg(p.absmax_q + b)) : __float_as_uint(__ldg(p.absmax + b));
      };
      auto load_codes = [&](int k) -> Codes { return load_codes64(p.codes + uint64_t(chunk_at(k)) * 32u, p.codes32 != 0); };
      const int first = (group + kDeqGroups - base % kDeqGroups) % kDeqGroups;
      uint32_t raw0 = raw_scale(first), raw1 = raw_scale(first + kDeqGroups);
      // Forward: a row's codes run along it, so four steps share a line and each
      // thread loads its own a step ahead.  dx walks down the rows: there the same
      // loads took 430 us against 405 through TMA (4096 x 11008, 4096 rows), and
      // the forward 665 us against 703 (11008 x 4096, 8192 rows).
      Codes next;
      if (MODE == kFwd) next = load_codes(first);
      for (int k = first; k < steps; k += kDeqGroups) {
        const uint32_t raw = raw0;
        raw0 = raw1;
        raw1 = raw_scale(k + 2 * kDeqGroups);
        const bool main = k < p.main_steps;
        uint4 v[8];
        Codes codes;
        if (MODE == kFwd) {
          codes = next;
          next = load_codes(k + kDeqGroups);
        } else if (main) {
          const int slot = kStages == kCodeSlots ? s : own_slot;
          ok = warp_wait(&sh->cfull[slot], (cph >> slot) & 1u, abort_flag, p.status);
          if (!ok) break;
          cph ^= 1u << slot;
          const uint8_t* src = code_base + slot * kCodeBytes;
          const uint32_t off = code_offset(uint32_t(row));
          const uint4 c0 = *reinterpret_cast<const uint4*>(src + off), c1 = *reinterpret_cast<const uint4*>(src + (off ^ 16u));
          codes = Codes{{c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w}};
        }
        if (main) {
          const float scale = k < k_end ? (dq ? __fmul_rn(float(raw), s_g) : __uint_as_float(raw)) : 0.0f;
          decode_row(codes, make_table(scale, F16), v);
        }
        ok = warp_wait(&sh->empty[s], ph, abort_flag, p.status);
        if (!ok) break;
        if (main) {
          uint8_t* tile = stage_w(s);
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(tile + sw128_offset(uint32_t(row), uint32_t(c))) = v[c];
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          arrive_leader(leader_bar(&sh->full[s]));   // adapter steps too: the same arrivals every phase
          // The code slot is given back only now: the stores above needed its codes
          // in registers.  Given back right after the loads were issued, the next
          // box could land before a load waiting behind other warps' stores.
          if (MODE == kDx && main) mbar_arrive(&sh->cempty[kStages == kCodeSlots ? s : own_slot]);
        }
        s += kDeqGroups;
        if (s >= kStages) {
          s -= kStages;
          ph ^= 1;
        }
        own_slot += kDeqGroups;
        if (own_slot >= kCodeSlots) own_slot -= kCodeSlots;
      }
      base += steps;
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side

PerDeviceOnce g_attr_done;

cudaError_t set_attrs() {
  const int dev = PerDeviceOnce::current();
  if (g_attr_done.done(dev)) return cudaSuccess;
  const void* kernels[] = {
      (const void*)expert_gemm_kernel<kFwd, false, 1>, (const void*)expert_gemm_kernel<kFwd, true, 1>,
      (const void*)expert_gemm_kernel<kFwd, false, 2>, (const void*)expert_gemm_kernel<kFwd, true, 2>,
      (const void*)expert_gemm_kernel<kDx, false, 1>,  (const void*)expert_gemm_kernel<kDx, true, 1>,
      (const void*)expert_gemm_kernel<kDx, false, 2>,  (const void*)expert_gemm_kernel<kDx, true, 2>,
      (const void*)expert_gemm_kernel<kI8, false, 1>};
  cudaError_t e = cudaSuccess;
  for (const void* k : kernels)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(std::max(gemm_smem(kDx, 1), gemm_smem(kDx, 2))));
  if (e == cudaSuccess) g_attr_done.mark(dev);
  return e;
}

bool set_grid(ExpertGemm* L, int sms) {
  ExpertParams& p = L->p;
  p.col_tiles = int((int64_t(p.out_cols) + kTileW - 1) / kTileW);
  const int64_t tiles = max_row_tiles(p.M, p.E, L->parts * kPartT) * p.col_tiles;
  if (tiles > int64_t(0x7fffffff)) return false;
  L->grid = 2u * unsigned(std::min<int64_t>(tiles, std::max(sms / 2, 1)));
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

template <int MODE, bool F16, int PARTS>
cudaError_t launch(const ExpertGemm& L, int prof_id, cudaStream_t st, int* launches) {
  cudaError_t e = set_attrs();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L.grid, 1, 1);
  cfg.blockDim = dim3(threads_of(MODE, PARTS), 1, 1);
  cfg.dynamicSmemBytes = gemm_smem(MODE, PARTS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = prof_on() ? 0 : 1;
  NF4_PROF_BEGIN(st, prof_id);
  e = cudaLaunchKernelEx(&cfg, expert_gemm_kernel<MODE, F16, PARTS>, L.maps, L.p);
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
  // Two MMAs a decoded weight tile where experts have more rows than one MMA
  // takes and one-MMA tiles would need a second wave of CTA pairs: a wide tile
  // costs 1.3 times a narrow one.  Measured, narrow against wide, 4096 x 4096:
  // 8 experts of 272 rows 132 us against 102, of 512 rows 138 against 117, of 240
  // rows 80 against 80; 2 experts of 1024 rows 78 against 64, but of 512 rows, 64
  // narrow tiles on 74 pairs, 48 against 61.
  const int64_t out_tiles = ((backward ? a.K : a.N) + kTileW - 1) / kTileW;
  parts = a.M > int64_t(kPartT) * g.E && a.M / kPartT * out_tiles > sms / 2 ? 2 : 1;
  ExpertGemm* L = this;
  const uint64_t N = uint64_t(a.N), K = uint64_t(a.K), E = uint64_t(g.E);
  const CUtensorMapSwizzle s128 = CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = token_maps(L, backward ? a.dy : a.x, backward ? N : K, ad, a.r, uint64_t(a.M));
  // a step's codes in dx: 128 columns of 64 W rows
  L->maps.w = L->maps.tok_l;
  if (backward)
    ok = ok && encode_map_stack(&L->maps.w, a.w->codes, MapElem::kU8, K / 2, N, E, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B);
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
  p.block_chunks_shift = log2_block(a.w->block_size) - 6;
  p.dq = a.w->double_quant;
  p.offsets = g.offsets;
  p.codes = a.w->codes;
  p.codes32 = (reinterpret_cast<uintptr_t>(a.w->codes) & 31u) == 0;
  p.absmax_q = a.w->absmax_q;
  p.absmax = a.w->absmax;
  p.absmax_scale = a.w->absmax_scale;
  p.bias = backward ? nullptr : a.bias;
  p.out = backward ? a.dx : a.y;
  p.status = a.status;
  // chunks are counted in 32 bits: stacks of up to 2.7e11 elements
  return ok && N * E * (K / 64) <= 0xffffffffull && set_grid(L, sms);
}

cudaError_t ExpertGemm::run(cudaStream_t st, int* launches) const {
  const int id = dx ? kKGroupedDx : kKGroupedFwd;
  if (parts == 2) {
    if (dx) return f16 ? launch<kDx, true, 2>(*this, id, st, launches) : launch<kDx, false, 2>(*this, id, st, launches);
    return f16 ? launch<kFwd, true, 2>(*this, id, st, launches) : launch<kFwd, false, 2>(*this, id, st, launches);
  }
  if (dx) return f16 ? launch<kDx, true, 1>(*this, id, st, launches) : launch<kDx, false, 1>(*this, id, st, launches);
  return f16 ? launch<kFwd, true, 1>(*this, id, st, launches) : launch<kFwd, false, 1>(*this, id, st, launches);
}

bool Int8Gemm::prepare(const Int8LinearArgs& a, int sms) {
  ExpertGemm& L = g;
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
  return ok && set_grid(&L, sms);
}

cudaError_t Int8Gemm::run(cudaStream_t st, int* launches) const {
  return launch<kI8, false, 1>(g, kKInt8Linear, st, launches);
}

}  // namespace nf4
