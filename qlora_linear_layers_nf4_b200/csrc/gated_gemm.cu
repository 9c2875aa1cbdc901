// The big products of the gated feed-forward layer on the sm_100a tensor cores:
//   kFwd   g = x W'_g^T + T_g B_g^T (+ bias), u = x W'_u^T + T_u B_u^T (+ bias), h = act(g) u
//   kDx    dx = dg W'_g + du W'_u + U_g A_g + U_u A_u
//
// As in the expert GEMM the weight is the A operand of the MMA (its outputs on the TMEM
// lanes), tokens are the B operand in even tiles of up to two MMAs of 256 (parts), so that
// a weight is decoded once for 512 tokens, and CTAs work in pairs (cta_group::2, M = 256).
//
// kFwd takes 128 outputs of both projections a tile: lane 2 i of a CTA's 128 holds row i of
// the gate's weight and lane 2 i + 1 row i of the up projection's, so g and u of an output
// lie in neighbouring lanes and one shuffle brings them together in the epilogue (the even
// lane takes the even tokens, the odd one the odd tokens).  The token tile is read once for
// both.  The adapter's steps walk T_g, then T_u; the weight side of a step is B's rows on
// that projection's lanes and zeros on the others, written by the dequant warps.
//
// kDx is one accumulation over both projections: first dg against the gate's weight, then
// du against the up projection's, then the two adapters.
//
// Roles in each CTA: warp 0 token TMA, warp 1 weight-side TMA (kDx), warp 2 MMA (issued by
// the pair's leader), from warp 4 on one or two epilogue groups, then the dequant groups.
// Rings: six stages of [weight tile 16 KB | tokens 16 KB], or four with 32 KB of tokens; six
// code slots (kDx); two accumulators of 256 TMEM columns.
//
// Bound by power back to back and by the MMAs' operand traffic alone: 4,096 tokens through
// 11008 x 4096, r = 64 (739 GFLOP), take 550 us forward (1.34 PFLOP/s; 576 with g, u and T
// stored) and 512 dx (1.44), tensor pipe 65 and 71 % active.  With few tokens a forward step takes
// 460 ns whatever they are: 64 tokens through the same layer 53 us, tensor pipe 11 %, DRAM 12 %,
// ALU and shared memory 44 %, issue 36 %; the dequant threads wait for their codes.
//
// Operands are of the compute type, so T, dg, du and U enter rounded to it once, as in the dense
// layer.  Their second terms would double the MMAs of dx and of the adapters; without them dx is
// off by 2.3e-3 (bf16) and 2.9e-4 (f16) relative to 64 bits where fp32 operands give 1.7e-3 and
// 2.1e-4, half a step of the result alone.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gated.h"
#include "gated_act.cuh"
#include "gated_rank.h"
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

constexpr int kFwd = 0;
constexpr int kDx = 1;

constexpr int kPartT = kGatedPartT;         // tokens of one MMA at most, half in each CTA
constexpr uint32_t kWBytes = 128 * 128;     // weight tile of a CTA: 128 x 128 bytes
constexpr uint32_t kTBytes = 128 * 128;     // its tokens of one part
constexpr uint32_t kCodeBytes = 128 * 32;   // kDx: NF4 codes of one step
constexpr int kCodeSlots = 6;
constexpr int kEpiWarp = 4;

constexpr int tile_w(int mode) { return gated_tile_w(mode == kDx); }   // outputs of a pair's tile
constexpr int stages_of(int parts) { return parts == 2 ? 4 : 6; }
// Dequant groups of four warps each take every deq_groups-th step; the stages and
// the code slots are multiples of their number, so that each belongs to one group.
constexpr int deq_groups(int parts) { return parts == 2 ? 2 : 3; }
// Epilogue groups of four warps.  The forward's epilogue (an exponential and a reciprocal an
// output) cannot run under the next tile's MMAs where a tile fills both accumulators: two
// groups take its pieces in turn.
constexpr int epi_groups(int mode, int parts) { return mode == 0 && parts == 2 ? 2 : 1; }
constexpr int deq_warp(int mode, int parts) { return kEpiWarp + 4 * epi_groups(mode, parts); }
constexpr int threads_of(int mode, int parts) { return 32 * (deq_warp(mode, parts) + 4 * deq_groups(parts)); }
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
};

// Behind the ring: kDx the code slots, kFwd two sets of staged pieces (h, g, u).
constexpr uint32_t kPiece = 32 * 128;
constexpr uint32_t extra_bytes(int mode) { return mode == kDx ? kCodeSlots * kCodeBytes : 2 * 3 * kPiece; }
constexpr size_t gemm_smem(int mode, int parts) {
  return size_t(stages_of(parts)) * stage_bytes_of(parts) + extra_bytes(mode) + sizeof(GemmShared) + 1024;
}
static_assert(gemm_smem(kDx, 1) <= 232448 && gemm_smem(kDx, 2) <= 232448 && gemm_smem(kFwd, 1) <= 232448 &&
                  gemm_smem(kFwd, 2) <= 232448,
              "shared memory of one CTA");

struct Tile {
  int k0, k1;   // its steps: all of them, or a split's
  int split;
  int t0, cnt;  // first token, tokens
  int nt[2];    // MMA columns of the parts (multiples of 16, of a first of two of 32; 0: no second part)
  int n0;       // first output
};

// Tile `id`, ordered by output tile, then token tile (then split): the pairs that run together
// share weight tiles and tokens.
template <int MODE, int PARTS>
__device__ __forceinline__ Tile tile_at(const GatedParams& p, int id) {
  Tile t;
  const int steps = p.main_steps + 2 * p.ad_steps;
  t.split = 0;
  t.k0 = 0;
  t.k1 = steps;
  if (p.splits > 1) {
    t.split = id % p.splits;
    id /= p.splits;
    t.k0 = steps * t.split / p.splits;
    t.k1 = steps * (t.split + 1) / p.splits;
  }
  const int ct = id / p.row_tiles, rt = id - ct * p.row_tiles;
  t.t0 = rt * p.tile_rows;
  t.cnt = min(p.tile_rows, p.M - t.t0);
  const int nt = (t.cnt + 15) & ~15;
  t.nt[0] = PARTS == 2 && nt > kPartT ? ((nt >> 1) + 31) & ~31 : nt;
  t.nt[1] = nt - t.nt[0];
  t.n0 = ct * tile_w(MODE);
  return t;
}

// kDx: byte offset in a step's code slot (64 reduction rows of 64 bytes, 64-byte swizzle)
// of the first of the two 16-byte chunks that weight-tile row `row` needs; the second is at
// that offset ^ 16.
__device__ __forceinline__ uint32_t code_offset(uint32_t row) {
  const uint32_t R = row & 63u, c = 2u * (row >> 6);
  return R * 64u + ((c ^ ((R >> 1) & 3u)) << 4);
}

// Sixteen values a lane, of tokens 2 j + (lane & 1) and output `out` of a CTA's 64, into a
// staged piece [32 tokens][64 outputs] (128-byte swizzle): lanes two apart (neighbouring
// outputs) trade so that each writes two outputs of a token.
template <bool F16>
__device__ __forceinline__ void stage_pairs(const float (&v)[16], uint8_t* piece, int out) {
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 2;
  const uint32_t first = uint32_t(lane & 1) + (hi ? 2u : 0u);
  const uint32_t chunk = uint32_t(out) >> 3, in = (uint32_t(out) & 6u) * 2u;
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float got = __shfl_xor_sync(0xffffffffu, hi ? v[j] : v[j + 1], 2);
    const uint32_t two = pack2(F16, hi ? got : v[j], hi ? v[j + 1] : got);
    *reinterpret_cast<uint32_t*>(piece + sw128_offset(first + 2u * uint32_t(j), chunk) + in) = two;
  }
}

// Tiled store of a 3-D box.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

template <int MODE, bool F16, int PARTS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(MODE, PARTS), 1)
    gated_gemm_kernel(const __grid_constant__ GatedMaps maps, const GatedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = expert::align_1024(smem_raw);
  constexpr int kStages = stages_of(PARTS);
  constexpr int kDeqGroups = deq_groups(PARTS);
  constexpr int kEpiGroups = epi_groups(MODE, PARTS);
  constexpr int kDeqWarp = deq_warp(MODE, PARTS);
  static_assert(kStages % kDeqGroups == 0 && kCodeSlots % kDeqGroups == 0, "a stage and a slot belong to one group");
  constexpr uint32_t kStageBytes = stage_bytes_of(PARTS);
  uint8_t* code_base = smem + kStages * kStageBytes;
  GemmShared* sh = reinterpret_cast<GemmShared*>(code_base + extra_bytes(MODE));
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
      mbar_init(&sh->full[s], 1 + 8);
      mbar_init(&sh->empty[s], 1);
    }
    for (int s = 0; s < kCodeSlots; ++s) {
      mbar_init(&sh->cfull[s], 1);
      mbar_init(&sh->cempty[s], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], 8 * kEpiGroups);   // leader: the epilogue warps of both CTAs
    }
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch(&maps.tok_l);
    tma_prefetch(&maps.tok_s);
    if (MODE == kFwd) tma_prefetch(&maps.h);
  }
  if (warp == 2) {
    tmem_alloc_pair(&sh->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int tiles = p.row_tiles * p.col_tiles * p.splits;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto leader_bar = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };
  // projection and first index within it of a main step, and of an adapter step
  auto main_proj = [&](int k) { return MODE == kDx && k >= p.half_steps ? 1 : 0; };
  auto ad_proj = [&](int k) { return k - p.main_steps >= p.ad_steps ? 1 : 0; };
  auto ad_r0 = [&](int k) { return (k - p.main_steps - (ad_proj(k) ? p.ad_steps : 0)) * 64; };

  // With two epilogue groups the 20 warps of 96 registers share them as 4 x 56 (loads, MMA),
  // 8 x 88 (epilogue) and 8 x 120 (dequant).
  constexpr bool kShare = kEpiGroups == 2;
  auto few_registers = [] {
    if constexpr (kShare) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  };

  // The single-issuer roles run as whole warps with one elected lane, so that
  // their counters and addresses stay in uniform registers.
  if (warp == 0) {
    few_registers();
    // ---------------- tokens: this CTA's half of the tile, in a 128-row box (or
    // a 32-row one)
    const bool issue = elect_one();
    // kDx: dg and du come from the kernels before, kFwd's T too
    bool waited = MODE == kDx, ok = true;
    if (MODE == kDx) {
      grid_dep_wait();
      // The gradients, launched behind this kernel, read nothing of it: they may fill the SMs
      // that it leaves free, now that what they read is complete.
      grid_dep_launch();
    }
    int s = 0, issued = 0;
    uint32_t ph = 1;
    for (int id = pair; id < tiles && ok; id += pairs) {
      const Tile t = tile_at<MODE, PARTS>(p, id);
      const int half = t.nt[0] >> 1;
      const bool large = half > 32;
      const bool two = PARTS == 2 && t.nt[1] > 0;
      const uint32_t bytes = two ? 2 * kTBytes : large ? kTBytes : 32u * 128u;   // of one CTA
      const int y = t.t0 + int(rank) * half;
      const int y2 = t.t0 + t.nt[0] + int(rank) * (t.nt[1] >> 1);
      const CUtensorMap* tok = large ? &maps.tok_l : &maps.tok_s;
      const CUtensorMap* ad = large ? &maps.ad_l : &maps.ad_s;
      for (int k = t.k0; k < t.k1; ++k) {
        ok = ring_wait(&sh->empty[s], ph, abort_flag, p.status);
        if (!ok) break;
        const bool main = k < p.main_steps;
        if (!main && !waited) grid_dep_wait();     // T: the kernel before
        waited |= !main;
        if (issue) {
          const uint32_t bar = leader_bar(&sh->full[s]);
          const bool w_tma = MODE == kDx && !main;   // the adapter's weight side
          if (rank == 0) mbar_arrive_expect_tx(&sh->full[s], 2 * (bytes + (w_tma ? kWBytes : 0u)));
          const int z = main ? main_proj(k) : ad_proj(k);
          const int x0 = main ? (k - (z ? p.half_steps : 0)) * 64 : ad_r0(k);
          tma_load_3d_pair(stage_t(s), main ? tok : ad, bar, x0, y, z);
          if (two) tma_load_3d_pair(stage_t(s) + kTBytes, main ? tok : ad, bar, x0, y2, z);
          if (w_tma) {
            const int n0 = t.n0 + 128 * int(rank);
            tma_load_3d_pair(stage_w(s), &maps.wad, bar, n0, x0, z);
            tma_load_3d_pair(stage_w(s) + 8192, &maps.wad, bar, n0 + 64, x0, z);
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
    // What runs after this grid may count on the kernel before it being done.
    if (!waited) grid_dep_wait();
    if (*abort_flag)   // unwind: wait (bounded) for the stages in flight
      for (int j = max(0, issued - kStages); j < issued; ++j) {
        uint32_t none = 0;
        ring_wait(&sh->empty[j % kStages], (j / kStages) & 1, &none, nullptr);
      }
  } else if (warp == 1) {
    // ---------------- kDx: the codes of every main step
    few_registers();
    if (MODE == kDx) {
      const bool issue = elect_one();
      int s = 0;
      uint32_t ph = (1u << kCodeSlots) - 1;   // bit s: parity of the wait for slot s, toggled at each use
      bool ok = true;
      for (int id = pair; id < tiles && ok; id += pairs) {
        const Tile t = tile_at<MODE, PARTS>(p, id);
        const int n0 = t.n0 + 128 * int(rank);
        for (int k = t.k0; k < t.k1; ++k) {
          if (k < p.main_steps) {
            ok = ring_wait(&sh->cempty[s], (ph >> s) & 1u, abort_flag, p.status);
            if (!ok) break;
            ph ^= 1u << s;
            if (issue) {
              const int z = main_proj(k);
              mbar_arrive_expect_tx(&sh->cfull[s], kCodeBytes);
              tma_load_2d(code_base + s * kCodeBytes, &maps.codes[z], &sh->cfull[s], n0 / 2, (k - (z ? p.half_steps : 0)) * 64);
            }
            __syncwarp();
          }
          if (++s == kCodeSlots) s = 0;
        }
      }
      if (*abort_flag)   // unwind: wait (bounded) for the codes in flight
        for (int j = 0; j < kCodeSlots; ++j) {
          uint32_t none = 0;
          ring_wait(&sh->cfull[j], (ph >> j) & 1u, &none, nullptr);
        }
    }
  } else if (warp == 2) {
    // ---------------- MMA: the leader's warp walks the steps, one lane issues
    few_registers();
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
        const Tile t = tile_at<MODE, PARTS>(p, id);
        const int parts = PARTS == 2 && t.nt[1] > 0 ? 2 : 1;
        for (int k = t.k0; k < t.k1 && ok; ++k) {
          ok = mbar_wait_cluster(&sh->full[s], ph, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t wd = w_desc + uint32_t(s) * (kStageBytes >> 4);
          const int left = k < p.main_steps ? 64 : p.r - ad_r0(k);
#pragma unroll
          for (int h = 0; h < PARTS; ++h) {
            if (h >= parts) break;
            const int b = (n + h) & 1;
            if (k == t.k0) {
              ok = mbar_wait_cluster(&sh->acc_empty[b], (((n + h) >> 1) & 1) ^ 1, abort_flag, p.status);
              if (!ok) break;
              tc_fence_after();
            }
            const uint32_t d = tmem + uint32_t(b) * 256u;
            const uint32_t idesc = idesc_f32acc(256, t.nt[h], MODE == kDx, false, F16);
            const uint64_t td = t_desc + uint32_t(s) * (kStageBytes >> 4) + uint32_t(h) * (kTBytes >> 4);
            if (issue) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk * 16 < left) umma_f16_pair(d, wd + kk * kWSub, td + kk * kTSub, idesc, (k > t.k0 || kk > 0) ? 1u : 0u);
              // The last step's commits go to the accumulators' barriers; the
              // epilogue then releases that step's stage.  MMAs finish in order,
              // so a commit covers the whole accumulation.
              if (k + 1 == t.k1) umma_commit_pair_mc(&sh->acc_full[b], 0x3);
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
  } else if (warp == 3) {
    few_registers();
  } else if (warp < kDeqWarp) {
    // ---------------- epilogue: lane = output (kFwd: projection lane & 1 of output
    // lane >> 1), register = token
    if constexpr (kShare) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int quad = warp & 3, group = (warp - kEpiWarp) >> 2;
    const int odd = lane & 1;
    int n = 0, last = 0;   // last: stage of the tile's last step
    [[maybe_unused]] int pieces = 0;   // kFwd: stored so far
    bool ok = true;
    for (int id = pair; id < tiles && ok; id += pairs) {
      const Tile t = tile_at<MODE, PARTS>(p, id);
      const int col = MODE == kFwd ? t.n0 + 64 * int(rank) + quad * 16 + (lane >> 1)
                                   : t.n0 + 128 * int(rank) + quad * 32 + lane;
      const bool col_ok = col < p.out_cols;
      float bias = 0.0f;
      if (MODE == kFwd && p.bias != nullptr && col_ok) {
        const int64_t at = int64_t(odd) * p.out_cols + col;
        bias = F16 ? __half2float(static_cast<const __half*>(p.bias)[at])
                   : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[at]);
      }
      last = (last + t.k1 - t.k0) % kStages;
      const int parts = PARTS == 2 && t.nt[1] > 0 ? 2 : 1;
#pragma unroll 1
      for (int h = 0; h < PARTS; ++h, ++n) {
        if (h >= parts) break;
        const int t0 = h == 0 ? t.t0 : t.t0 + t.nt[0];
        const int cnt = h + 1 == parts ? t.t0 + t.cnt - t0 : t.nt[0];
        ok = warp_wait<300>(&sh->acc_full[n & 1], (n >> 1) & 1, abort_flag, p.status);
        if (MODE == kFwd) ok = named_barrier_and(1 + group, 128, ok);   // the warps that store together go on together
        if (!ok) break;
        if (h + 1 == parts && group == 0 && quad == 0 && lane == 0) mbar_arrive(&sh->empty[(last + kStages - 1) % kStages]);
        tc_fence_after();
#pragma unroll 1
        for (int c = group; c * 32 < cnt; c += kEpiGroups) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + uint32_t(n & 1) * 256u + c * 32, v);
          tmem_ld_wait();
          const int left = cnt - c * 32;
          const int64_t row0 = int64_t(t0) + c * 32;
          if (MODE == kFwd) {
            if (PARTS == 1 && p.splits > 1) {   // fp32 sums of the split, added up by the kernel after
              float* o = p.partials + ((int64_t(t.split) * p.M + row0) * 2 + odd) * p.out_cols + col;
#pragma unroll
              for (int i = 0; i < 32; ++i, o += 2 * int64_t(p.out_cols))
                if (col_ok && i < left) __stcg(o, __uint_as_float(v[i]));
              continue;
            }
            float g[16], u[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float a = __uint_as_float(v[i]) + bias, b = __uint_as_float(v[i + 1]) + bias;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
              g[i / 2] = odd ? got : a;
              u[i / 2] = odd ? b : got;
            }
            // Pieces [32 tokens][64 outputs] of the group's four warps leave by TMA as whole
            // lines.  (As 32-byte pieces straight from
            // registers the forward of 4096 tokens with g and u took 728 us against 600
            // without.)
            constexpr int kSets = kEpiGroups == 2 ? 1 : 2;   // of a group
            uint8_t* piece = code_base + (group + pieces % kSets) * (3 * kPiece);
            if (pieces >= kSets) {   // the stores of kSets pieces ago have read this set
              if (quad == 0 && lane == 0) bulk_wait_group_read<kSets - 1>();
              named_barrier(1 + group, 128);
            }
            ++pieces;
            const int out = quad * 16 + (lane >> 1);
            const bool pre = p.pre != nullptr;
            if (pre) {
              stage_pairs<F16>(g, piece + kPiece, out);
              stage_pairs<F16>(u, piece + 2 * kPiece, out);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] = gated::act<true>(p.act, g[i]) * u[i];
            stage_pairs<F16>(g, piece, out);
            fence_proxy_async_smem();
            named_barrier(1 + group, 128);
            if (quad == 0 && lane == 0) {
              const int x0 = t.n0 + 64 * int(rank);
              if (x0 < p.out_cols) {   // outputs past N and tokens past M are clipped
                tma_store_3d(&maps.h, piece, x0, int(row0), 0);
                if (pre) {
                  tma_store_3d(&maps.pre, piece + kPiece, x0, int(row0), 0);
                  tma_store_3d(&maps.pre, piece + 2 * kPiece, x0, int(row0), 1);
                }
              }
              bulk_commit_group();
            }
          } else {
            if (PARTS == 1 && p.splits > 1) {   // likewise
              float* o = p.partials + (int64_t(t.split) * p.M + row0) * p.out_cols + col;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (col_ok && i < left) __stcg(o + int64_t(i) * p.out_cols, __uint_as_float(v[i]));
              continue;
            }
            // two lanes trade so that each stores two neighbouring outputs of one token
            uint16_t* o = static_cast<uint16_t*>(p.out) + (row0 + odd) * p.out_cols + (col & ~1);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float a = __uint_as_float(v[i]), b = __uint_as_float(v[i + 1]);
              const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
              const uint32_t two = pack2(F16, odd ? got : a, odd ? b : got);
              if (col_ok && i + odd < left) *reinterpret_cast<uint32_t*>(o + int64_t(i) * p.out_cols) = two;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(leader_bar(&sh->acc_empty[n & 1]));
      }
    }
    if (MODE == kFwd && quad == 0 && lane == 0) bulk_wait_group_all();
  } else if (warp >= kDeqWarp) {
    // ---------------- dequant warps: one thread per weight-tile row and step, so
    // the table of a block's sixteen values is built once.  A group of four warps
    // takes every kDeqGroups-th step: decoding (codes to registers) needs no free
    // stage, so it runs ahead of the MMAs, and only the stores wait for the stage.
    if constexpr (kShare) asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    const int group = (warp - kDeqWarp) >> 2;
    const int row = threadIdx.x & 127;
    const bool dq = p.dq != 0;
    // kFwd: a row's projection is fixed.  kDx: that of the step.
    const int rp = MODE == kFwd ? row & 1 : 0;
    float s_g[2];
    s_g[0] = dq ? __ldg(p.absmax_scale[rp]) : 0.0f;
    s_g[1] = dq && MODE == kDx ? __ldg(p.absmax_scale[1]) : s_g[0];
    const uint32_t per_row = uint32_t(p.w_cols) >> 6;
    int base = 0;                // steps of the tiles before
    int s = group;               // stage of this group's next step
    uint32_t ph = 1;             // parity of the wait for that stage
    int own_slot = group;        // and its code slot (with as many stages as slots: the stage's)
    uint32_t cph = 0;            // bit i: parity of the wait for the codes in slot i
    bool ok = true;
    for (int id = pair; id < tiles && ok; id += pairs) {
      const Tile t = tile_at<MODE, PARTS>(p, id);
      // this row's 64-element chunk at step k of its projection: c0 + k * c_step; its scale
      // is that of the block that holds it
      const int wr0 = MODE == kFwd ? t.n0 + 64 * int(rank) + (row >> 1) : row & 63;
      const int ch0 = MODE == kFwd ? 0 : ((t.n0 + 128 * int(rank)) >> 6) + (row >> 6);
      const uint32_t c0 = uint32_t(wr0) * per_row + uint32_t(ch0);
      const uint32_t c_step = MODE == kFwd ? 1u : 64u * per_row;
      // rows past the weight decode to zeros: their scale counts as 0 (and their loads read
      // the last row that is there, or the first)
      const int k_end = MODE == kFwd ? (wr0 < p.w_rows ? p.half_steps : 0)
                                     : (uint32_t(ch0) < per_row ? (p.w_rows - wr0 + 63) >> 6 : 0);
      const uint32_t c_base = k_end > 0 ? c0 : 0u;
      auto step_in = [&](int k) { return MODE == kDx && k >= p.half_steps ? k - p.half_steps : k; };
      auto chunk_at = [&](int k) { return c_base + uint32_t(max(min(step_in(k), k_end - 1), 0)) * c_step; };
      // Scales are loaded two of this thread's steps ahead and converted only
      // where they are used, so that no step waits for a load.
      auto raw_scale = [&](int k) -> uint32_t {
        const uint32_t b = chunk_at(k) >> p.block_chunks_shift;
        const int z = MODE == kFwd ? rp : main_proj(k);
        return dq ? uint32_t(__ldg(p.absmax_q[z] + b)) : __float_as_uint(__ldg(p.absmax[z] + b));
      };
      auto load_codes = [&](int k) -> Codes {
        return load_codes64(p.codes[rp] + uint64_t(chunk_at(k)) * 32u, p.codes32[rp] != 0);
      };
      const int first = t.k0 + (group + kDeqGroups - base % kDeqGroups) % kDeqGroups;
      uint32_t raw0 = raw_scale(first), raw1 = raw_scale(first + kDeqGroups);
      Codes next;
      if (MODE == kFwd) next = load_codes(first);
      for (int k = first; k < t.k1; k += kDeqGroups) {
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
          const float scale = step_in(k) < k_end ? (dq ? __fmul_rn(float(raw), s_g[main_proj(k)]) : __uint_as_float(raw)) : 0.0f;
          decode_row(codes, make_table(scale, F16), v);
        } else if (MODE == kFwd) {
          // the adapter's rows of this projection, zeros elsewhere (r % 8 == 0: whole chunks)
          const int z = ad_proj(k), r0 = ad_r0(k);
          const bool mine = z == rp && wr0 < p.w_rows;
          const uint4* b = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.B) + (int64_t(z) * p.w_rows + (mine ? wr0 : 0)) * p.r + r0);
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = mine && r0 + 8 * c < p.r ? __ldg(b + c) : make_uint4(0u, 0u, 0u, 0u);
        }
        ok = warp_wait(&sh->empty[s], ph, abort_flag, p.status);
        if (!ok) break;
        if (main || MODE == kFwd) {
          uint8_t* tile = stage_w(s);
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(tile + sw128_offset(uint32_t(row), uint32_t(c))) = v[c];
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          arrive_leader(leader_bar(&sh->full[s]));   // kDx's adapter steps too: the same arrivals every phase
          // The code slot is given back only now: the stores above needed its codes
          // in registers.
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
      base += t.k1 - t.k0;
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

constexpr int kSumThreads = 256;

// Four values of every split, added up in their order.
__device__ __forceinline__ float4 sum4(const float* __restrict__ parts, int splits, int64_t stride) {
  float4 v = __ldcg(reinterpret_cast<const float4*>(parts));
  for (int s = 1; s < splits; ++s) {
    const float4 w = __ldcg(reinterpret_cast<const float4*>(parts + int64_t(s) * stride));
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  }
  return v;
}
template <bool F16>
__device__ __forceinline__ uint2 round4(float4 v) {
  return make_uint2(pack2(F16, v.x, v.y), pack2(F16, v.z, v.w));
}

// h, and g and u, from the splits' sums [split][M][2][N]: four outputs a thread.
template <bool F16>
__global__ void __launch_bounds__(kSumThreads) gated_finish_kernel(const GatedParams p) {
  const int64_t n = int64_t(p.M) * p.out_cols;
  uint16_t* h = static_cast<uint16_t*>(p.out);
  uint16_t* pre = static_cast<uint16_t*>(p.pre);
  for (int64_t i = (int64_t(blockIdx.x) * kSumThreads + threadIdx.x) * 4; i < n; i += int64_t(gridDim.x) * kSumThreads * 4) {
    const int64_t row = i / p.out_cols;
    const int col = int(i - row * p.out_cols);
    float4 v[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      v[z] = sum4(p.partials + (2 * row + z) * p.out_cols + col, p.splits, 2 * n);
      if (p.bias != nullptr) {
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.bias) + int64_t(z) * p.out_cols + col));
        const float2 lo = unpack2(F16, b.x), hi = unpack2(F16, b.y);
        v[z] = make_float4(v[z].x + lo.x, v[z].y + lo.y, v[z].z + hi.x, v[z].w + hi.y);
      }
      if (pre != nullptr) *reinterpret_cast<uint2*>(pre + z * n + i) = round4<F16>(v[z]);
    }
    *reinterpret_cast<uint2*>(h + i) =
        round4<F16>(make_float4(gated::act<true>(p.act, v[0].x) * v[1].x, gated::act<true>(p.act, v[0].y) * v[1].y,
                                gated::act<true>(p.act, v[0].z) * v[1].z, gated::act<true>(p.act, v[0].w) * v[1].w));
  }
}

// dx from the splits' sums: four outputs a thread.
template <bool F16>
__global__ void __launch_bounds__(kSumThreads) gated_sum_kernel(const float* __restrict__ parts, int splits, int64_t n, uint16_t* __restrict__ out) {
  for (int64_t i = (int64_t(blockIdx.x) * kSumThreads + threadIdx.x) * 4; i < n; i += int64_t(gridDim.x) * kSumThreads * 4) {
    *reinterpret_cast<uint2*>(out + i) = round4<F16>(sum4(parts + i, splits, n));
  }
}

// ------------------------------------------------------------------ host side

PerDeviceOnce g_attr_done;

cudaError_t set_attrs() {
  const int dev = PerDeviceOnce::current();
  if (g_attr_done.done(dev)) return cudaSuccess;
  const void* kernels[] = {
      (const void*)gated_gemm_kernel<kFwd, false, 1>, (const void*)gated_gemm_kernel<kFwd, true, 1>,
      (const void*)gated_gemm_kernel<kFwd, false, 2>, (const void*)gated_gemm_kernel<kFwd, true, 2>,
      (const void*)gated_gemm_kernel<kDx, false, 1>,  (const void*)gated_gemm_kernel<kDx, true, 1>,
      (const void*)gated_gemm_kernel<kDx, false, 2>,  (const void*)gated_gemm_kernel<kDx, true, 2>};
  cudaError_t e = cudaSuccess;
  for (const void* k : kernels)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(std::max(std::max(gemm_smem(kDx, 1), gemm_smem(kDx, 2)), std::max(gemm_smem(kFwd, 1), gemm_smem(kFwd, 2)))));
  if (e == cudaSuccess) g_attr_done.mark(dev);
  return e;
}

template <int MODE, bool F16, int PARTS>
cudaError_t launch(const GatedGemm& L, cudaStream_t st, int* launches) {
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
  const int id = MODE == kDx ? kKGatedDx : kKGatedFwd;
  NF4_PROF_BEGIN(st, id);
  e = cudaLaunchKernelEx(&cfg, gated_gemm_kernel<MODE, F16, PARTS>, L.maps, L.p);
  NF4_PROF_END(st, id);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <int MODE>
cudaError_t launch_mode(const GatedGemm& L, cudaStream_t st, int* launches) {
  if (L.parts == 2) return L.f16 ? launch<MODE, true, 2>(L, st, launches) : launch<MODE, false, 2>(L, st, launches);
  return L.f16 ? launch<MODE, true, 1>(L, st, launches) : launch<MODE, false, 1>(L, st, launches);
}

// T [2][M][r], or the first of each projection's terms of U [2][terms][M][r].
bool ad_map(CUtensorMap* map, const void* ad, uint64_t r, uint64_t M, uint64_t terms, uint32_t box_rows) {
  const uint64_t dims[3] = {r, M, 2}, strides[2] = {r * 2, terms * M * r * 2};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_map(map, ad, MapElem::k16, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

bool GatedGemm::prepare(const GatedArgs& a, bool backward, const void* tok, const void* ad, void* scratch, int sms) {
  dx = backward;
  f16 = a.f16 != 0;
  const uint64_t M = uint64_t(a.M), N = uint64_t(a.N), K = uint64_t(a.K), r = uint64_t(a.r);
  const GatedGemmPlan plan = gated_gemm_plan(backward, a.M, a.N, a.K, a.r, sms);
  parts = plan.parts;
  const CUtensorMapSwizzle s128 = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t depth = backward ? 2 : 1, cols = backward ? N : K;
  const uint64_t ad_terms = backward ? uint64_t(gated_terms(f16)) : 1;
  bool ok = encode_map_stack(&maps.tok_l, tok, MapElem::k16, cols, M, depth, 64, 128, s128) &&
            encode_map_stack(&maps.tok_s, tok, MapElem::k16, cols, M, depth, 64, 32, s128) &&
            ad_map(&maps.ad_l, ad, r, M, ad_terms, 128) && ad_map(&maps.ad_s, ad, r, M, ad_terms, 32);
  maps.wad = maps.codes[0] = maps.codes[1] = maps.h = maps.pre = maps.tok_l;
  if (!backward) {
    ok = ok && encode_map_stack(&maps.h, a.h, MapElem::k16, N, M, 1, 64, 32, s128);
    if (a.pre_out != nullptr) ok = ok && encode_map_stack(&maps.pre, a.pre_out, MapElem::k16, N, M, 2, 64, 32, s128);
  }
  if (backward) {
    ok = ok && encode_map_stack(&maps.wad, a.A, MapElem::k16, K, r, 2, 64, 64, s128);
    for (int i = 0; i < 2; ++i)   // a step's codes: 128 columns of 64 W rows
      ok = ok && encode_map_2d(&maps.codes[i], a.w[i]->codes, MapElem::kU8, K / 2, N, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  p = GatedParams{};
  p.M = int(a.M);
  p.out_cols = int(backward ? a.K : a.N);
  p.w_rows = int(a.N);
  p.w_cols = int(a.K);
  p.r = a.r;
  p.half_steps = plan.half_steps;
  p.main_steps = plan.main_steps;
  p.ad_steps = plan.ad_steps;
  p.col_tiles = plan.col_tiles;
  p.row_tiles = plan.row_tiles;
  p.tile_rows = plan.tile_rows;
  p.splits = plan.splits;
  p.block_chunks_shift = log2_block(a.w[0]->block_size) - 6;
  p.dq = a.w[0]->double_quant;
  p.act = a.act;
  for (int i = 0; i < 2; ++i) {
    p.codes[i] = a.w[i]->codes;
    p.codes32[i] = (reinterpret_cast<uintptr_t>(a.w[i]->codes) & 31u) == 0;
    p.absmax_q[i] = a.w[i]->absmax_q;
    p.absmax[i] = a.w[i]->absmax;
    p.absmax_scale[i] = a.w[i]->absmax_scale;
  }
  p.B = a.B;
  p.bias = backward ? nullptr : a.bias;
  p.out = backward ? a.dx : a.h;
  p.pre = backward ? nullptr : a.pre_out;
  p.status = a.status;
  p.partials = static_cast<float*>(scratch);
  grid = 2u * unsigned(plan.pairs);
  // chunks are counted in 32 bits: weights of up to 2.7e11 elements
  return ok && N * (K / 64) <= 0xffffffffull && plan.tiles <= int64_t(0x7fffffff);
}

cudaError_t GatedGemm::sum(cudaStream_t st, int* launches) const {
  if (p.splits == 1) return cudaSuccess;
  const int64_t n = int64_t(p.M) * p.out_cols;   // a multiple of 8
  const unsigned ctas = unsigned(std::min<int64_t>((n / 4 + kSumThreads - 1) / kSumThreads, 4096));
  const int id = dx ? kKGatedDx : kKGatedFwd;
  NF4_PROF_BEGIN(st, id);
  if (!dx && f16) gated_finish_kernel<true><<<ctas, kSumThreads, 0, st>>>(p);
  else if (!dx) gated_finish_kernel<false><<<ctas, kSumThreads, 0, st>>>(p);
  else if (f16) gated_sum_kernel<true><<<ctas, kSumThreads, 0, st>>>(p.partials, p.splits, n, static_cast<uint16_t*>(p.out));
  else gated_sum_kernel<false><<<ctas, kSumThreads, 0, st>>>(p.partials, p.splits, n, static_cast<uint16_t*>(p.out));
  NF4_PROF_END(st, id);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t GatedGemm::run(cudaStream_t st, int* launches) const {
  return dx ? launch_mode<kDx>(*this, st, launches) : launch_mode<kFwd>(*this, st, launches);
}

}  // namespace nf4
