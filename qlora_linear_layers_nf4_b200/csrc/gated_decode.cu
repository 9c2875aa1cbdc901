// Forward of the gated layer for a few tokens (serving steps): both 4-bit weights are
// streamed once.
//
//   g[m, n] = sum_k W'_gate[n, k] x[m, k] + sum_j T_0[m, j] B_0[n, j] (+ bias_0[n]),  u likewise,
//   h[m, n] = act(g) u
//
// The kernel is the expert layer's weight-streaming one (expert_decode.cu) with tiles that
// hold 64 outputs of both projections: 128 weight rows, a unit of work 256 columns of them
// (16 KB of codes); every SM has the same number of whole tiles, and before them a share of
// the tiles that are left over.  A warp takes 8 gate rows as the
// MMA rows 0 .. 7 and the same 8 up rows as 8 .. 15, so a thread that finishes a gate row has
// the up row of its output in the next lane.  A quarter of the weights, half of the gate's,
// are decoded with byte permutes, the others with shared-memory lookups (44032 x 4096 and one
// token: half and half 77 us, a quarter 72, an eighth 73, none 76.5); the adapters' products
// are two MMAs, T_0 with the up rows zero and T_1 with the gate rows zero.
//
// Bound by decoding: four instructions a weight; at 44032 x 4096 (one token, 16 tokens) shared
// memory is 74 and 77 % busy, the byte-permute pipe 57 and 51 %, issue 57 and 54 %, DRAM 31 and 27 %.
// Two weights of 11008 x 4096 (47 MB) take 23 to 24 us with one token (2.0 TB/s), 29 with 16, of
// which 8 to 9 are start and T, whose CTAs hold SMs whole (equal shares of all units, with the join
// of split tiles at their end: 27 and 33).  A unit, 256 columns of a tile, takes a CTA 1 us.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_common.cuh"
#include "gated_act.cuh"
#include "gated_decode.h"
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
constexpr int kDcOutputs = kGatedDecodeOutputs;       // of a tile, a gate and an up row each
static_assert(2 * kDcOutputs == kDcRows, "a row a thread");
constexpr int kDcBlocks = kGatedDecodeChunk / 64;    // 64-wide K blocks per unit
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
};
template <int NP>
constexpr size_t dc_smem() {
  return size_t(dc_stages(NP)) * dc_stage_bytes(NP) + kLutBytes + sizeof(DcShared<NP>) + 1024;
}
static_assert(dc_smem<16>() <= 232448 && dc_smem<8>() <= 232448, "shared memory of one CTA");

// A tile of the work list: token group and 64 outputs.  The roles walk the tiles of a share
// one after another.
struct DcTile {
  int rt, nt;
};
__device__ __forceinline__ DcTile dc_tile(int n_tiles, uint32_t tile) {
  DcTile t;
  t.rt = int(tile / uint32_t(n_tiles));
  t.nt = int(tile) - t.rt * n_tiles;
  return t;
}
__device__ __forceinline__ void dc_next(int n_tiles, DcTile& t) {
  if (++t.nt < n_tiles) return;
  t.nt = 0;
  ++t.rt;
}

template <int NP, bool F16>
__global__ void __launch_bounds__(kDcThreads, 1)
    gated_decode_kernel(const __grid_constant__ CUtensorMap tm_gate, const __grid_constant__ CUtensorMap tm_up,
                        const __grid_constant__ CUtensorMap tm_x, const GatedDecodeParams p) {
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
    tma_prefetch(&tm_gate);
    tma_prefetch(&tm_up);
    tma_prefetch(&tm_x);
  }
  __syncthreads();

  // Work of a CTA: a share of the first `rest` tiles, then `whole` tiles of its own.  Of those
  // first tiles CTA c of G takes units [units c / G, units (c + 1) / G); tiles that so fall to
  // several CTAs are joined while their last contributor's own tiles still run.
  const uint32_t kch = uint32_t(p.k_chunks);
  const uint32_t units = uint32_t(p.rest) * kch;     // < 2^31, as all tiles' units are
  const uint32_t G = uint32_t(p.rest_ctas);
  const bool shares = blockIdx.x < G;
  const uint32_t share0 = shares ? uint32_t(uint64_t(units) * blockIdx.x / G) : 0u;
  const uint32_t share1 = shares ? uint32_t(uint64_t(units) * (blockIdx.x + 1) / G) : 0u;
  const uint32_t own0 = (uint32_t(p.rest) + blockIdx.x * uint32_t(p.whole)) * kch, own1 = own0 + uint32_t(p.whole) * kch;
  struct Range {
    uint32_t u0, u1, tile0;
    int kc0;      // the range's first chunk of its first tile
    int group0;   // the group that takes its first unit: groups take a CTA's units in turn
  };
  auto range_at = [&](int i) {
    Range r;
    r.u0 = i ? own0 : share0;
    r.u1 = i ? own1 : share1;
    r.tile0 = r.u0 / kch;
    r.kc0 = int(r.u0 - r.tile0 * kch);
    r.group0 = i ? int((share1 - share0) % kGroups) : 0;
    return r;
  };

  if (warp == kProducer) {
    // ---------------- producer
    int s = 0, issued = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int i = 0; i < 2 && ok; ++i) {
      const Range r = range_at(i);
      DcTile t = dc_tile(p.n_tiles, r.tile0);
      int kc = r.kc0;
      for (uint32_t u = r.u0; u < r.u1; ++u) {
        ok = warp_wait(&sh->empty[s], ph, abort_flag, p.status);
        if (!ok) break;
        if (lane == 0) {
          uint8_t* dst = smem + s * dc_stage_bytes(NP);
          mbar_arrive_expect_tx(&sh->full[s], dc_stage_bytes(NP));
          tma_load_2d(dst, &tm_gate, &sh->full[s], kc * 128, t.nt * kDcOutputs);
          tma_load_2d(dst + kDcCodeBytes / 2, &tm_up, &sh->full[s], kc * 128, t.nt * kDcOutputs);
          tma_load_3d(dst + kDcCodeBytes, &tm_x, &sh->full[s], 0, t.rt * NP, kc * kDcBlocks);
        }
        __syncwarp();
        if (++kc == p.k_chunks) {
          kc = 0;
          dc_next(p.n_tiles, t);
        }
        ++issued;
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (*abort_flag)   // unwind: wait (bounded) for the boxes in flight
      for (int j = max(0, issued - kStages); j < issued; ++j) {
        uint32_t none = 0;
        ring_wait(&sh->full[j % kStages], (j / kStages) & 1, &none, nullptr);
      }
    return;
  }

  if (warp >= kScaler) {
    // ---------------- scales of a group's units: loaded a unit ahead, stored when
    // the stage is free
    const int group = warp - kScaler;
    const bool dq = p.dq != 0;
    const float s_g[2] = {dq ? __ldg(p.absmax_scale[0]) : 0.0f, dq ? __ldg(p.absmax_scale[1]) : 0.0f};
    const int kb_per_row = p.K >> 6;
    // Block 64 and whole chunks: a row's four scales of a unit are one aligned word or vector.
    const bool vec = p.vec_scales != 0;
    uint4 raw[4];
    auto load_scales = [&](const DcTile& t, int kc) {   // outputs lane and lane + 32, of the gate, then up
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = min(t.nt * kDcOutputs + 32 * (i & 1) + lane, p.N - 1);
        const int64_t at = int64_t(n) * p.K + int64_t(kc) * (64 * kDcBlocks);
        const uint8_t* absmax_q = p.absmax_q[i >> 1];
        const float* absmax = p.absmax[i >> 1];
        if (vec) {
          if (dq) raw[i].x = __ldg(reinterpret_cast<const uint32_t*>(absmax_q + (at >> 6)));
          else raw[i] = __ldg(reinterpret_cast<const uint4*>(absmax + (at >> 6)));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t b = (at + min(j, kb_per_row - 1 - kc * kDcBlocks) * 64) >> p.bs_shift;
            w[j] = dq ? uint32_t(__ldg(absmax_q + b)) : __float_as_uint(__ldg(absmax + b));
          }
          raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    int s = group;
    uint32_t ph = 1;
    bool ok = true;
    for (int i = 0; i < 2 && ok; ++i) {
      const Range r = range_at(i);
      const uint32_t first = uint32_t((group + kGroups - r.group0) % kGroups);
      if (r.u0 + first >= r.u1) continue;
      DcTile t = dc_tile(p.n_tiles, r.tile0);
      int kc = r.kc0 + int(first);
      auto settle = [&]() {   // (t, kc) to the tile that holds the chunk
        while (kc >= p.k_chunks) {
          kc -= p.k_chunks;
          dc_next(p.n_tiles, t);
        }
      };
      settle();
      load_scales(t, kc);
      for (uint32_t u = r.u0 + first; u < r.u1; u += kGroups) {
        uint4 now[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) now[i] = raw[i];
        if (u + kGroups < r.u1) {
          kc += kGroups;
          settle();
          load_scales(t, kc);
        }
        ok = warp_wait(&sh->empty[s], ph, abort_flag, p.status);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
          if (vec && dq) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = (now[i].x >> (8 * j)) & 0xffu;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sh->scales[s][j][2 * (32 * (i & 1) + lane) + (i >> 1)] = dq ? __fmul_rn(float(w[j]), s_g[i >> 1]) : __uint_as_float(w[j]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->full[s]);
        s += kGroups;
        if (s >= kStages) {
          s -= kStages;
          ph ^= 1;
        }
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
    for (int i = 0; i < 2; ++i) {
      const Range r = range_at(i);
      DcTile t = dc_tile(p.n_tiles, r.tile0);
      uint32_t tile_u = r.tile0 * kch;          // first unit of the tile, in whatever CTA
      for (uint32_t u = r.u0; u < r.u1; tile_u += kch, dc_next(p.n_tiles, t)) {
        const bool starts = u == tile_u;        // this CTA has the tile's first chunk
        const uint32_t end = min(r.u1, tile_u + kch);
        const bool split = end - u < kch;
        u = end;
        const int rows = min(NP, p.M - t.rt * NP);
        const int n = t.nt * kDcOutputs + (row >> 1);
        if (starts) {
          const uint16_t* b = p.B + (int64_t(row & 1) * p.N + min(n, p.N - 1)) * p.r;
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
#pragma unroll 2
            for (uint32_t c = c0; c <= c1; ++c) {
              const float* part = p.partials + (size_t(c) * 2 + (c == c0 ? 1 : 0)) * (kDcRows * NP) + row;
#pragma unroll
              for (int m = 0; m < NP; ++m)
                if (m < rows) v[m] += __ldcg(part + m * kDcRows);
            }
          }
        }
        // Lanes 2 i and 2 i + 1 hold g and u of one output: the even lane takes the even
        // tokens, the odd one the odd tokens.
        if (finish && ok) {
          const int odd = row & 1;
          const bool there = n < p.N;
          const float bias = there && p.bias != nullptr ? one_float<F16>(__ldg(p.bias + int64_t(odd) * p.N + n)) : 0.0f;
#pragma unroll
          for (int m = 0; m < NP; m += 2) {
            const float a = v[m] + bias, b = v[m + 1] + bias;
            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
            const float g = odd ? got : a, u = odd ? b : got;
            if (!there || m + odd >= rows) continue;
            const int64_t at = int64_t(t.rt * NP + m + odd) * p.N + n;
            p.h[at] = one_rounded<F16>(gated::act<true>(p.act, g) * u);
            if (p.pre != nullptr) {
              p.pre[at] = one_rounded<F16>(g);
              p.pre[int64_t(p.M) * p.N + at] = one_rounded<F16>(u);
            }
          }
        }
        named_barrier(1, kEpi);   // red and last may be written again
        if (lane == 0) mbar_arrive(&sh->red_free);
      }
    }
    if (!waited) grid_dep_wait();
    return;
  }

  // ---------------- consumers
  // A warp takes 8 outputs of a unit, their gate rows as the MMA rows g and their up rows as
  // g + 8.  The four lanes of an output take a 64-wide block each, whole: the k index of an
  // MMA is free as long as W' and x agree, so lane q's four k positions are columns of block
  // q.  Half of the gate's row is decoded with byte permutes from a table of its block's
  // sixteen products (as in the GEMM), the rest with the shared-memory lookups.
  //
  // Lookup table: byte (even element in the high nibble) -> two levels, one copy per lane.  It
  // is made while the first loads are on their way (before the roles part it cost 0.6 us more).
  uint32_t my = 0;
#pragma unroll
  for (int c = 0; c < 16; ++c) my = (lane & 15) == c ? level_bits(c) : my;
  const float lv = __uint_as_float(my);
  for (int e = warp; e < 256; e += kConsumers) {
    const float hi = __shfl_sync(0xffffffffu, lv, e >> 4);
    const float lo = __shfl_sync(0xffffffffu, lv, e & 15);
    reinterpret_cast<float2*>(lut)[e * 32 + lane] = make_float2(hi, lo);
  }
  named_barrier(2, 32 * kConsumers);

  const int group = warp / kDcGroupWarps;
  const int set = warp % kDcGroupWarps;     // outputs 8 set ..
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
    const uint32_t row = uint32_t(i * kDcOutputs + set * 8 + g);
    code_at[i] = row * 128u + ((uint32_t(2 * q + (q >> 1)) ^ (row & 7u)) << 4) + (uint32_t(q & 1) << 3);
  }
  const uint32_t x_at = kDcCodeBytes + uint32_t(q) * (NP * 128) + uint32_t(g) * 128u + (uint32_t((2 * q) ^ g) << 4);
  for (int part = 0; part < 2; ++part) {
    const Range r = range_at(part);
    DcTile t = dc_tile(p.n_tiles, r.tile0);
    int kc = r.kc0 + (group + kGroups - r.group0) % kGroups;   // chunk of this warp's next unit, counted from tile t
    uint32_t tile_u = r.tile0 * kch;
    for (uint32_t seg = r.u0; seg < r.u1; tile_u += kch, dc_next(p.n_tiles, t)) {
      const bool first_part = seg == tile_u;
      seg = min(r.u1, tile_u + kch);
      const int kend = int(seg - tile_u);     // this CTA's chunks of the tile end here
      float acc[2][NT8][4];                   // of even and odd MMAs
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < NT8; ++c) acc[i][c][0] = acc[i][c][1] = acc[i][c][2] = acc[i][c][3] = 0.0f;
      for (; kc < kend; kc += kGroups) {
        if (ok && !__all_sync(0xffffffffu, mbar_try_wait(&sh->full[s], ph))) ok = warp_wait(&sh->full[s], ph, abort_flag, p.status);
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
              const uint2 lo = expert::decode4(c0 & 0x7777u, ((c0 >> 1) & 0x4444u) | 0x3210u, table);
              const uint4 v = make_uint4(lo.x, lo.y, two_weights<2, F16>(lut, c0, lane8, scale.x), two_weights<3, F16>(lut, c0, lane8, scale.x));
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

      // The adapters' products enter the tile's first part, as MMAs with the rows of B as A
      // (of one projection, the other's zero) and T as B; the groups take 32 columns in turn,
      // a lane eight consecutive ones of its rows in a load (two at a time were 45.7 us against
      // 34.7 with 16 tokens and r = 64).
      if (first_part) {
        if (!waited) grid_dep_wait();   // T of the kernel before
        waited = true;
        const int n = min(t.nt * kDcOutputs + set * 8 + g, p.N - 1);
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        for (int j = 32 * group + 8 * q; j - 8 * q < p.r; j += 32 * kGroups) {   // r is a multiple of 8
          const bool there = j < p.r;
          uint4 bv[2], tv[2][NT8];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            bv[z] = there ? __ldg(reinterpret_cast<const uint4*>(p.B + (int64_t(z) * p.N + n) * p.r + j)) : none;
#pragma unroll
            for (int c = 0; c < NT8; ++c) {
              const int m = t.rt * NP + 8 * c + g;
              tv[z][c] = there && m < p.M ? __ldcg(reinterpret_cast<const uint4*>(p.T + (int64_t(z) * p.M + m) * p.r + j)) : none;
            }
          }
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t lo[4] = {0u, 0u, 0u, 0u}, hi[4] = {0u, 0u, 0u, 0u};
            lo[z] = bv[z].x, lo[2 + z] = bv[z].y, hi[z] = bv[z].z, hi[2 + z] = bv[z].w;
#pragma unroll
            for (int c = 0; c < NT8; ++c) {
              mma_16816<F16>(acc[0][c], lo, tv[z][c].x, tv[z][c].y);
              mma_16816<F16>(acc[0][c], hi, tv[z][c].z, tv[z][c].w);
            }
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
}

// T_p = s x A_p^T of a few tokens.  A CTA takes eight adapter rows and sixteen tokens; its
// 32 warps share the columns in pieces of 32, a lane eight of them of its row of A and of two
// tokens (an MMA's k positions are free as long as both operands agree), and their fp32 sums
// are joined in a fixed order.  It is latency that counts: all loads of a row of 4096 are on
// their way at once, and the few CTAs leave the other SMs to the decode kernel, which starts
// beside them.  (A CTA of eight warps for each adapter row and eight tokens, summing products
// of fp32, read x once per adapter row: a call of 16 tokens with r = 64 took 52.6 us against
// 45.7, of 8 with r = 16 34.1 against 30.0.)  Also clears the decode kernel's counters.
constexpr int kTsWarps = 32;
constexpr int kTsRows = 8;
constexpr int kTsTokens = 16;
template <bool F16>
__global__ void __launch_bounds__(32 * kTsWarps, 1)
    gated_t_small_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ A, int M, int K, int r, float scale,
                         uint16_t* __restrict__ T, int* counters, int n_counters) {
  __shared__ float part[kTsWarps][kTsTokens * kTsRows];
  grid_dep_launch();
  const int j0 = blockIdx.x * kTsRows, m0 = blockIdx.y * kTsTokens;   // j0: of both projections' rows
  if (blockIdx.x == 0 && m0 == 0)
    for (int i = threadIdx.x; i < n_counters; i += 32 * kTsWarps) counters[i] = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const bool there[2] = {m0 + g < M, m0 + g + 8 < M};
  const uint16_t* a = A + int64_t(j0 + g) * K + 8 * q;
  const uint16_t* x0 = x + int64_t(m0 + g) * K + 8 * q;
  const uint16_t* x1 = x0 + int64_t(8) * K;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  float acc[2][4] = {};
#pragma unroll 4
  for (int k = 32 * warp; k < K; k += 32 * kTsWarps) {
    const uint4 av = __ldg(reinterpret_cast<const uint4*>(a + k));
    const uint4 u = there[0] ? __ldg(reinterpret_cast<const uint4*>(x0 + k)) : none;
    const uint4 v = there[1] ? __ldg(reinterpret_cast<const uint4*>(x1 + k)) : none;
    const uint32_t lo[4] = {u.x, v.x, u.y, v.y}, hi[4] = {u.z, v.z, u.w, v.w};
    mma_16816<F16>(acc[0], lo, av.x, av.y);
    mma_16816<F16>(acc[1], hi, av.z, av.w);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<float2*>(&part[warp][(g + 8 * i) * kTsRows + 2 * q]) =
        make_float2(acc[0][2 * i] + acc[1][2 * i], acc[0][2 * i + 1] + acc[1][2 * i + 1]);
  __syncthreads();
  const int m = m0 + int(threadIdx.x) / kTsRows, j = j0 + int(threadIdx.x) % kTsRows;
  if (threadIdx.x < kTsTokens * kTsRows && m < M) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kTsWarps; ++w) v += part[w][threadIdx.x];
    const int z = j >= r ? 1 : 0;
    T[(int64_t(z) * M + m) * r + j - z * r] = one_rounded<F16>(scale * v);
  }
}

PerDeviceOnce g_attr_done;

cudaError_t set_attrs() {
  const int dev = PerDeviceOnce::current();
  if (g_attr_done.done(dev)) return cudaSuccess;
  const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(gated_decode_kernel<8, false>, attr, int(dc_smem<8>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gated_decode_kernel<8, true>, attr, int(dc_smem<8>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gated_decode_kernel<16, false>, attr, int(dc_smem<16>()));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gated_decode_kernel<16, true>, attr, int(dc_smem<16>()));
  if (e == cudaSuccess) g_attr_done.mark(dev);
  return e;
}

template <int NP, bool F16>
cudaError_t launch(const GatedDecode& L, cudaStream_t st) {
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
  return cudaLaunchKernelEx(&cfg, gated_decode_kernel<NP, F16>, L.codes[0], L.codes[1], L.x, L.p);
}

}  // namespace

size_t gated_decode_scratch_bytes() { return size_t(kGatedDecodeMaxCtas) * (2 * kDcRows * 16 * sizeof(float) + 16); }

bool GatedDecode::prepare(const GatedArgs& a, const void* T, uint8_t* scratch, int sms) {
  const GatedDecodePlan plan = gated_decode_plan(a.M, a.N, a.K, sms);
  np = plan.np;
  f16 = a.f16 != 0;
  const uint64_t K = uint64_t(a.K), N = uint64_t(a.N), M = uint64_t(a.M), kb = K / 64;
  bool ok = true;
  for (int z = 0; z < 2; ++z)
    ok = ok && encode_map_2d(&codes[z], a.w[z]->codes, MapElem::kU8, K / 2, N, 128, kDcOutputs, CU_TENSOR_MAP_SWIZZLE_128B);
  {  // x as [K blocks][tokens][64]
    const uint64_t dims[3] = {64, M, kb}, strides[2] = {K * 2, 128};
    const uint32_t box[3] = {64, uint32_t(np), uint32_t(kDcBlocks)};
    ok = ok && encode_map(&x, a.x, MapElem::k16, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  p = GatedDecodeParams{};
  p.M = int(a.M);
  p.N = int(a.N);
  p.K = int(a.K);
  p.r = a.r;
  p.n_tiles = plan.n_tiles;
  p.k_chunks = plan.k_chunks;
  p.row_tiles = plan.row_tiles;
  p.whole = plan.whole;
  p.rest = plan.rest;
  p.rest_ctas = plan.rest_ctas;
  p.bs_shift = log2_block(a.w[0]->block_size);
  p.dq = a.w[0]->double_quant;
  p.act = a.act;
  for (int z = 0; z < 2; ++z) {
    p.absmax_q[z] = a.w[z]->absmax_q;
    p.absmax[z] = a.w[z]->absmax;
    p.absmax_scale[z] = a.w[z]->absmax_scale;
  }
  p.B = static_cast<const uint16_t*>(a.B);
  p.T = static_cast<const uint16_t*>(T);
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.h = static_cast<uint16_t*>(a.h);
  p.pre = static_cast<uint16_t*>(a.pre_out);
  p.partials = reinterpret_cast<float*>(scratch);
  p.counters = reinterpret_cast<int*>(scratch + size_t(kGatedDecodeMaxCtas) * 2 * kDcRows * 16 * sizeof(float));
  p.status = a.status;
  p.vec_scales = a.w[0]->block_size == 64 && a.K % 256 == 0;   // scale pointers are 16-byte aligned
  grid = unsigned(plan.ctas);
  return ok && plan.fits;
}

cudaError_t GatedDecode::run(cudaStream_t st, int* launches) const {
  cudaError_t e = set_attrs();
  if (e != cudaSuccess) return e;
  NF4_PROF_BEGIN(st, kKGatedFwd);
  if (np == 8) e = f16 ? launch<8, true>(*this, st) : launch<8, false>(*this, st);
  else e = f16 ? launch<16, true>(*this, st) : launch<16, false>(*this, st);
  NF4_PROF_END(st, kKGatedFwd);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_gated_t_small(const GatedArgs& a, void* T, int* counters, cudaStream_t st, int* launches) {
  const dim3 grid(unsigned(2 * a.r / kTsRows), unsigned((a.M + kTsTokens - 1) / kTsTokens), 1);
  const auto* x = static_cast<const uint16_t*>(a.x);
  const auto* A = static_cast<const uint16_t*>(a.A);
  auto* t = static_cast<uint16_t*>(T);
  const int n = counters != nullptr ? kGatedDecodeMaxCtas : 0;
  NF4_PROF_BEGIN(st, kKGatedT);
  if (a.f16)
    gated_t_small_kernel<true><<<grid, 32 * kTsWarps, 0, st>>>(x, A, int(a.M), int(a.K), a.r, a.s, t, counters, n);
  else
    gated_t_small_kernel<false><<<grid, 32 * kTsWarps, 0, st>>>(x, A, int(a.M), int(a.K), a.r, a.s, t, counters, n);
  NF4_PROF_END(st, kKGatedT);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nf4
