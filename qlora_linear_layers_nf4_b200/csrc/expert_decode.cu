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
// Inside a CTA two groups of eight warps take turns at the units (so that their
// waits, loads and MMAs overlap), a warp 16 rows.  W' is made in registers, as A
// fragments of mma.sync m16n8k16 with x as B, bit for bit the GEMM's: the fp32
// product of level and scale rounded to the compute type.  Two ways share the work,
// because each fills another pipe.  Half of the rows go through byte permutes on a
// table of their block's sixteen products, in registers; the other half looks a
// code byte up in a 256-entry table of fp32 level pairs, replicated per lane
// (conflict-free; entries 256 bytes apart, so that one byte permute makes the
// offset), and multiplies and rounds.  A 16-token step took 86 us so, 95 with the
// lookups alone (1,024 of a unit's 1,400 shared-memory wavefronts) and more with
// the permutes alone.  (Levels rounded to 16 bits in the table and the scale on the
// block's sums would be cheaper still, but made y's error 1.6 times as large.)
// A producer warp keeps code and x boxes in flight and a warp per group the scales
// of its units; four more warps finish a tile (sums, bias, split tiles) while the
// next one streams.  8 experts of 8192 x 4096 with 32 rows: 69 us for 143 MB; the
// pipe of byte permutes 63 %, issue 60 %, shared memory 46 %, DRAM 26 % of peak: the
// decoding of four warps a scheduler, between their waits, is what remains.
//
// T = s x A_e^T comes from a small kernel launched just before, which this one
// overlaps (programmatic dependent launch) until it finishes its first tile.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_common.cuh"
#include "expert_decode.h"
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
using namespace decode;
using expert::ring_wait;
using expert::warp_wait;

constexpr int kDcGroupWarps = 8;                     // 16 rows each
constexpr int kDcEpiWarps = 4;                       // finish tiles, a thread per row
constexpr int kDcRows = 32 * kDcEpiWarps;
constexpr int kDcBlocks = 4;                         // 64-wide K blocks per unit
constexpr uint32_t kDcCodeBytes = kDcRows * 128;
constexpr uint32_t kLutBytes = 256 * 256;            // entry e, lane l at 256 e + 8 l

// Groups of consumer warps, each with a scale warp (three groups of fewer registers
// were 5 % slower).
constexpr int kDcGroups = 2;
constexpr int kDcConsumers = kDcGroups * kDcGroupWarps;
constexpr int kDcThreads = 32 * (kDcConsumers + kDcEpiWarps + kDcGroups + 1);
// A multiple of the groups: a stage always belongs to the same one.
constexpr int dc_stages(int np) { return np == 8 ? 6 : 4; }
constexpr uint32_t dc_stage_bytes(int np) { return kDcCodeBytes + uint32_t(np) * 512u; }

template <int NP>
struct DcShared {
  uint64_t full[dc_stages(NP)];                      // boxes landed, scales written
  uint64_t empty[dc_stages(NP)];
  uint64_t red_full;                                 // the consumers have stored their sums of a tile
  uint64_t red_free;                                 // the finishing warps have read them
  uint32_t abort_flag;
  int last;                                          // this CTA finishes the tile
  float scales[dc_stages(NP)][kDcBlocks][kDcRows + 8];   // + 8: a warp's reads of four blocks hit different banks
  float red[kDcGroups][kDcRows * NP];        // the consumers' sums of a tile, [token][row]
  GroupTable groups;
};
template <int NP>
constexpr size_t dc_smem() {
  return size_t(dc_stages(NP)) * dc_stage_bytes(NP) + kLutBytes + sizeof(DcShared<NP>) + 1024;
}
static_assert(dc_smem<16>() <= 232448 && dc_smem<8>() <= 232448, "shared memory of one CTA");

// A tile of the work list: row group, its expert and first row, 128 W rows.  The
// roles walk the tiles of a share one after another.
struct DcTile {
  int rt, nt;
  int e, row0;
};
__device__ __forceinline__ void dc_expert(const GroupTable* g, int E, int np, DcTile& t) {
  t.e = expert_of_tile(g, E, t.rt);
  t.row0 = g->start[t.e] + (t.rt - g->tiles[t.e]) * np;
}
__device__ __forceinline__ DcTile dc_tile(const GroupTable* g, int E, int np, int n_tiles, uint32_t tile) {
  DcTile t;
  t.rt = int(tile / uint32_t(n_tiles));
  t.nt = int(tile) - t.rt * n_tiles;
  dc_expert(g, E, np, t);
  return t;
}
__device__ __forceinline__ void dc_next(const GroupTable* g, int E, int np, int n_tiles, DcTile& t) {
  if (++t.nt < n_tiles) return;
  t.nt = 0;
  if (++t.rt < g->tiles[E]) dc_expert(g, E, np, t);
}

template <int NP, bool F16>
__global__ void __launch_bounds__(kDcThreads, 1)
    expert_decode_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_x,
                         const DecodeParams p) {
  constexpr int kStages = dc_stages(NP);
  constexpr int kGroups = kDcGroups, kConsumers = kDcConsumers;
  constexpr int kScaler = kConsumers + kDcEpiWarps;  // first scale warp
  constexpr int kProducer = kScaler + kGroups;
  constexpr int NT8 = NP / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = expert::align_1024(smem_raw);
  uint8_t* lut = smem + kStages * dc_stage_bytes(NP);
  DcShared<NP>* sh = reinterpret_cast<DcShared<NP>*>(lut + kLutBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sh->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh->full[s], 2);   // the producer and the scale warp
      mbar_init(&sh->empty[s], kDcGroupWarps);
    }
    mbar_init(&sh->red_full, kConsumers);
    mbar_init(&sh->red_free, kDcEpiWarps);
    sh->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch(&tm_codes);
    tma_prefetch(&tm_x);
  }
  if (warp == kProducer) {
    build_groups(&sh->groups, p.offsets, p.E, p.M, NP, blockIdx.x == 0 ? p.status : nullptr);
  } else if (warp < kConsumers) {
    // Lookup table: byte (even element in the high nibble) -> two levels, one copy per lane.
    uint32_t my = 0;
#pragma unroll
    for (int c = 0; c < 16; ++c) my = (lane & 15) == c ? level_bits(c) : my;
    const float lv = __uint_as_float(my);
    for (int e = warp; e < 256; e += kConsumers) {
      const float hi = __shfl_sync(0xffffffffu, lv, e >> 4);
      const float lo = __shfl_sync(0xffffffffu, lv, e & 15);
      reinterpret_cast<float2*>(lut)[e * 32 + lane] = make_float2(hi, lo);
    }
  }
  __syncthreads();

  // Shares: CTA c of G takes units [units c / G, units (c + 1) / G).  G counts the
  // CTAs with work, at least one unit each.
  const GroupTable* groups = &sh->groups;
  const uint32_t kch = uint32_t(p.k_chunks);
  const uint32_t units = uint32_t(groups->tiles[p.E]) * uint32_t(p.n_tiles) * kch;   // < 2^31
  const uint32_t G = min(gridDim.x, units);
  const bool works = blockIdx.x < G;
  const uint32_t u0 = works ? uint32_t(uint64_t(units) * blockIdx.x / G) : 0u;
  const uint32_t u1 = works ? uint32_t(uint64_t(units) * (blockIdx.x + 1) / G) : 0u;
  const uint32_t tile0 = u0 / kch;
  const int kc0 = int(u0 - tile0 * kch);             // the share's first chunk of its first tile

  if (warp == kProducer) {
    // ---------------- producer
    if (u0 < u1) {
      DcTile t = dc_tile(groups, p.E, NP, p.n_tiles, tile0);
      int kc = kc0, s = 0, issued = 0;
      uint32_t ph = 1;
      for (uint32_t u = u0; u < u1; ++u) {
        if (!warp_wait(&sh->empty[s], ph, abort_flag, p.status)) break;
        if (lane == 0) {
          uint8_t* dst = smem + s * dc_stage_bytes(NP);
          mbar_arrive_expect_tx(&sh->full[s], dc_stage_bytes(NP));
          tma_load_3d(dst, &tm_codes, &sh->full[s], kc * 128, t.nt * kDcRows, t.e);
          tma_load_3d(dst + kDcCodeBytes, &tm_x, &sh->full[s], 0, t.row0, kc * kDcBlocks);
        }
        __syncwarp();
        if (++kc == p.k_chunks) {
          kc = 0;
          dc_next(groups, p.E, NP, p.n_tiles, t);
        }
        ++issued;
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (*abort_flag)   // unwind: wait (bounded) for the boxes in flight
        for (int j = max(0, issued - kStages); j < issued; ++j) {
          uint32_t none = 0;
          ring_wait(&sh->full[j % kStages], (j / kStages) & 1, &none, nullptr);
        }
    }
    return;
  }

  if (warp >= kScaler) {
    // ---------------- scales of a group's units: loaded a unit ahead, stored when
    // the stage is free
    const int group = warp - kScaler;
    const bool dq = p.dq != 0;
    const float s_g = dq ? __ldg(p.absmax_scale) : 0.0f;
    const int kb_per_row = p.K >> 6;
    // Block 64 and whole chunks: a row's four scales of a unit are one aligned word or vector.
    const bool vec = p.vec_scales != 0;
    uint4 raw[4];
    auto load_scales = [&](const DcTile& t, int kc) {   // rows lane, lane + 32, ...
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = min(t.nt * kDcRows + 32 * i + lane, p.N - 1);
        const int64_t at = (int64_t(t.e) * p.N + n) * p.K + int64_t(kc) * (64 * kDcBlocks);
        if (vec) {
          if (dq) raw[i].x = __ldg(reinterpret_cast<const uint32_t*>(p.absmax_q + (at >> 6)));
          else raw[i] = __ldg(reinterpret_cast<const uint4*>(p.absmax + (at >> 6)));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t b = (at + min(j, kb_per_row - 1 - kc * kDcBlocks) * 64) >> p.bs_shift;
            w[j] = dq ? uint32_t(__ldg(p.absmax_q + b)) : __float_as_uint(__ldg(p.absmax + b));
          }
          raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    DcTile t{};
    int kc = kc0 + group;
    auto settle = [&]() {   // (t, kc) to the tile that holds the chunk
      while (kc >= p.k_chunks) {
        kc -= p.k_chunks;
        dc_next(groups, p.E, NP, p.n_tiles, t);
      }
    };
    if (u0 + uint32_t(group) < u1) {
      t = dc_tile(groups, p.E, NP, p.n_tiles, tile0);
      settle();
      load_scales(t, kc);
    }
    int s = group;
    uint32_t ph = 1;
    for (uint32_t u = u0 + group; u < u1; u += kGroups) {
      uint4 now[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) now[i] = raw[i];
      if (u + kGroups < u1) {
        kc += kGroups;
        settle();
        load_scales(t, kc);
      }
      if (!warp_wait(&sh->empty[s], ph, abort_flag, p.status)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
        if (vec && dq) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = (now[i].x >> (8 * j)) & 0xffu;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sh->scales[s][j][32 * i + lane] = dq ? __fmul_rn(float(w[j]), s_g) : __uint_as_float(w[j]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->full[s]);
      s += kGroups;
      if (s >= kStages) {
        s -= kStages;
        ph ^= 1;
      }
    }
    return;
  }

  if (warp >= kConsumers) {
    // ---------------- finishing warps: a thread per row of the tile
    constexpr int kEpi = 32 * kDcEpiWarps;
    const int row = threadIdx.x - 32 * kConsumers;
    bool ok = true, waited = false;
    uint32_t ph = 0;
    DcTile t{};
    if (u0 < u1) t = dc_tile(groups, p.E, NP, p.n_tiles, tile0);
    uint32_t tile_u = tile0 * kch;            // first unit of the tile, in whatever CTA
    for (uint32_t u = u0; u < u1; tile_u += kch, dc_next(groups, p.E, NP, p.n_tiles, t)) {
      const bool starts = u == tile_u;        // this CTA has the tile's first chunk
      const uint32_t end = min(u1, tile_u + kch);
      const bool split = end - u < kch;
      u = end;
      const int rows = min(NP, groups->start[t.e + 1] - t.row0);
      const int64_t n0 = int64_t(t.e) * p.N;
      const int n = t.nt * kDcRows + row;
      if (starts) {
        const uint16_t* b = p.B + (n0 + min(n, p.N - 1)) * p.r;
        for (int j = 0; j < p.r; j += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(b + j));
      }
      if (!waited) grid_dep_wait();   // the counters' zeros, of the kernel before
      waited = true;
      if (ok) ok = warp_wait<100>(&sh->red_full, ph, abort_flag, p.status);
      ph ^= 1;
      float v[NP];
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        v[m] = 0.0f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) v[m] += sh->red[i][m * kDcRows + row];
      }
      bool finish = true;
      if (split) {
        // contributors are consecutive CTAs, the first from chunk 0
        const uint32_t c0 = uint32_t((uint64_t(tile_u + 1) * G - 1) / units);
        const uint32_t c1 = uint32_t((uint64_t(tile_u + kch) * G - 1) / units);
        float* mine = p.partials + (size_t(blockIdx.x) * 2 + (starts ? 1 : 0)) * (kDcRows * NP) + row;
#pragma unroll
        for (int m = 0; m < NP; ++m)
          if (m < rows) __stcg(mine + m * kDcRows, v[m]);
        __threadfence();
        named_barrier(1, kEpi);
        if (row == 0) sh->last = atomicAdd(p.counters + c0, 1) == int(c1 - c0);
        named_barrier(1, kEpi);
        finish = sh->last != 0;
        if (finish) {
          // a contributor's rows are loaded together: one after another they were a
          // tail of 13 us behind the last tile (a tenth of a 16-token step)
          __threadfence();
#pragma unroll
          for (int m = 0; m < NP; ++m) v[m] = 0.0f;
          for (uint32_t c = c0; c <= c1; ++c) {
            const float* part = p.partials + (size_t(c) * 2 + (c == c0 ? 1 : 0)) * (kDcRows * NP) + row;
#pragma unroll
            for (int m = 0; m < NP; ++m)
              if (m < rows) v[m] += __ldcg(part + m * kDcRows);
          }
        }
      }
      if (finish && ok && n < p.N) {
        const float bias = p.bias != nullptr ? one_float<F16>(__ldg(p.bias + n0 + n)) : 0.0f;
        uint16_t* y = p.y + int64_t(t.row0) * p.N + n;
#pragma unroll
        for (int m = 0; m < NP; ++m)
          if (m < rows) y[int64_t(m) * p.N] = one_rounded<F16>(v[m] + bias);
      }
      named_barrier(1, kEpi);   // red and last may be written again
      if (lane == 0) mbar_arrive(&sh->red_free);
    }
    if (!waited) grid_dep_wait();
    return;
  }

  // ---------------- consumers
  // A warp takes 16 W rows of a unit.  The four lanes of a row pair (2 g and 2 g + 1,
  // the MMA rows g and g + 8) take a 64-wide block each, whole: the k index of an MMA
  // is free as long as W' and x agree, so lane q's four k positions are columns of
  // block q.  Row 2 g is decoded with byte permutes from a table of its block's
  // sixteen products (as in the GEMM), row 2 g + 1 with the shared-memory lookups.
  const int group = warp / kDcGroupWarps;
  const int set = warp % kDcGroupWarps;     // rows 16 set ..
  const int g = lane >> 2, q = lane & 3;
  const uint32_t lane8 = uint32_t(lane) << 3;   // below 256: one byte
  const int kb_per_row = p.K >> 6;
  bool ok = true, waited = false;
  int s = group;
  uint32_t ph = 0, red_ph = 1;
  // Addresses inside a stage.  Lane q walks its block's 16-byte-of-x steps in the
  // order i ^ 2 q and its code granules in the order m ^ q, so that the lanes' loads
  // hit different banks.
  uint32_t code_at[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t row = uint32_t(set * 16 + 2 * g + i);
    code_at[i] = row * 128u + ((uint32_t(2 * q + (q >> 1)) ^ (row & 7u)) << 4) + (uint32_t(q & 1) << 3);
  }
  const uint32_t x_at = kDcCodeBytes + uint32_t(q) * (NP * 128) + uint32_t(g) * 128u + (uint32_t((2 * q) ^ g) << 4);
  DcTile t{};
  if (u0 < u1) t = dc_tile(groups, p.E, NP, p.n_tiles, tile0);
  int kc = kc0 + group;                     // chunk of this warp's next unit, counted from tile t
  uint32_t tile_u = tile0 * kch;
  for (uint32_t seg = u0; seg < u1; tile_u += kch, dc_next(groups, p.E, NP, p.n_tiles, t)) {
    const bool first_part = seg == tile_u;
    seg = min(u1, tile_u + kch);
    const int kend = int(seg - tile_u);     // this CTA's chunks of the tile end here
    float acc[2][NT8][4];                   // of even and odd MMAs
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < NT8; ++c) acc[i][c][0] = acc[i][c][1] = acc[i][c][2] = acc[i][c][3] = 0.0f;
    for (; kc < kend; kc += kGroups) {
      if (ok) ok = warp_wait(&sh->full[s], ph, abort_flag, p.status);
      if (ok) {
        const uint8_t* st = smem + s * dc_stage_bytes(NP);
        float2 scale = *reinterpret_cast<const float2*>(&sh->scales[s][q][set * 16 + 2 * g]);
        if (kc * kDcBlocks + q >= kb_per_row) scale = make_float2(0.0f, 0.0f);   // past the row's end: x is zero there
        const expert::BlockTable table = expert::make_table(scale.x, F16);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint2 w0 = *reinterpret_cast<const uint2*>(st + (code_at[0] ^ (m * 8u)));
          const uint2 w1 = *reinterpret_cast<const uint2*>(st + (code_at[1] ^ (m * 8u)));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t c0 = h ? w0.y : w0.x, c1 = h ? w1.y : w1.x;
            const uint4 v = expert::decode8(c0, table);
            const uint32_t a0[4] = {v.x, two_weights<0, F16>(lut, c1, lane8, scale.y), v.y, two_weights<1, F16>(lut, c1, lane8, scale.y)};
            const uint32_t a1[4] = {v.z, two_weights<2, F16>(lut, c1, lane8, scale.y), v.w, two_weights<3, F16>(lut, c1, lane8, scale.y)};
#pragma unroll
            for (int c = 0; c < NT8; ++c) {
              const uint4 xv = *reinterpret_cast<const uint4*>(st + (x_at ^ ((2 * m + h) * 16u)) + c * 1024);
              mma_16816<F16>(acc[0][c], a0, xv.x, xv.y);
              mma_16816<F16>(acc[1][c], a1, xv.z, xv.w);
            }
          }
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&sh->empty[s]);
      s += kGroups;
      if (s >= kStages) {
        s -= kStages;
        ph ^= 1;
      }
    }
    kc -= p.k_chunks;
#pragma unroll
    for (int c = 0; c < NT8; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[0][c][i] += acc[1][c][i];

    // The adapter's product enters the tile's first part, as MMAs with the rows
    // of B_e as A and T as B; the groups take 16 columns in turn.
    if (first_part) {
      if (!waited) grid_dep_wait();   // T of the kernel before
      waited = true;
      for (int j0 = 16 * group; j0 < p.r; j0 += 16 * kGroups) {
        const int ja = j0 + 2 * q, jb = ja + 8;   // r is a multiple of 8: the second half may be missing
        uint32_t a[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = min(t.nt * kDcRows + set * 16 + 2 * g + h, p.N - 1);
          const uint16_t* brow = p.B + (int64_t(t.e) * p.N + n) * p.r;
          a[h] = __ldg(reinterpret_cast<const uint32_t*>(brow + ja));
          a[2 + h] = jb < p.r ? __ldg(reinterpret_cast<const uint32_t*>(brow + jb)) : 0u;
        }
#pragma unroll
        for (int c = 0; c < NT8; ++c) {
          const int m = t.row0 + 8 * c + g;
          const uint16_t* trow = p.T + int64_t(min(m, p.M - 1)) * p.r;
          const uint32_t b0 = m < p.M ? __ldcg(reinterpret_cast<const uint32_t*>(trow + ja)) : 0u;
          const uint32_t b1 = m < p.M && jb < p.r ? __ldcg(reinterpret_cast<const uint32_t*>(trow + jb)) : 0u;
          mma_16816<F16>(acc[0][c], a, b0, b1);
        }
      }
    }

    // the tile's sums, for the finishing warps
    if (ok) ok = warp_wait(&sh->red_free, red_ph, abort_flag, p.status);
    red_ph ^= 1;
    const int row = set * 16 + 2 * g;
#pragma unroll
    for (int c = 0; c < NT8; ++c) {
      float* o = sh->red[group] + (8 * c + 2 * q) * kDcRows + row;
      *reinterpret_cast<float2*>(o) = make_float2(acc[0][c][0], acc[0][c][2]);
      *reinterpret_cast<float2*>(o + kDcRows) = make_float2(acc[0][c][1], acc[0][c][3]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->red_full);
  }
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
  // Rows of an expert per pass over its weight: 16 cost more a pass and save the
  // second pass of an expert with more than 8.  Measured, 8 against 16: 8 experts of
  // 4096 x 4096 with 4, 6 and 8 rows on average 43, 49 and 55.4 us against 51, 53 and
  // 54.4; 64 of 1024 x 2048 with 6 and 8 rows 52 and 59 against 54 and 54.
  np = a.M <= 8 || a.M <= 6 * int64_t(g.E) ? 8 : 16;
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
  p.vec_scales = a.w->block_size == 64 && a.K % 256 == 0;   // scale pointers are 16-byte aligned
  const int64_t most = max_row_tiles(a.M, g.E, np) * p.n_tiles * p.k_chunks;
  if (most > int64_t(0x7fffffff)) return false;
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
