// How a call of the gated layer is cut into work: which kernel takes it, its tiles and the splits
// of its reduction.  Host arithmetic alone (no CUDA), so that the tests can ask which form a size
// takes.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace nf4 {

constexpr int64_t plan_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- few tokens: both weights streamed (gated_decode.cu)

constexpr int kGatedDecodeMaxCtas = 160;      // most CTAs of a launch; sizes the scratch
constexpr int kGatedDecodeOutputs = 64;       // of a tile, a gate and an up row each
constexpr int kGatedDecodeChunk = 256;        // columns of a unit of work

struct GatedDecodePlan {
  int np;                   // tokens per group
  int row_tiles, n_tiles;   // groups of tokens, tiles of outputs
  int k_chunks;             // units of a tile
  int whole;                // tiles that a CTA has of its own, behind
  int rest, rest_ctas;      // the first tiles, which rest_ctas CTAs share
  int ctas;
  bool fits;                // units are counted in 31 bits
};

// Whole tiles for every SM, and the rest shared: where it leaves two SMs or more for a tile
// each has CTAs of its own, up to eight, as a share that straddles two tiles stores and joins
// parts of both (1000 x 4096: one token 15.6 -> 10.6 us, 16 tokens 28.5 -> 14.2; 4096 x 4096,
// 16 tokens: 20.6 -> 18.4).
inline GatedDecodePlan gated_decode_plan(int64_t M, int64_t N, int64_t K, int sms) {
  GatedDecodePlan p{};
  p.np = M <= 8 ? 8 : 16;
  p.row_tiles = int(plan_cdiv(M, p.np));
  p.n_tiles = int(plan_cdiv(N, kGatedDecodeOutputs));
  p.k_chunks = int(plan_cdiv(K, kGatedDecodeChunk));
  const int64_t tiles = int64_t(p.row_tiles) * p.n_tiles, ctas = std::min(sms, kGatedDecodeMaxCtas);
  p.fits = tiles * p.k_chunks <= int64_t(0x7fffffff);
  p.whole = int(tiles / ctas);
  p.rest = int(tiles % ctas);
  const int64_t each = p.rest > 0 ? std::min<int64_t>({8, ctas / p.rest, p.k_chunks}) : 0;
  p.rest_ctas = int(each >= 2 ? each * p.rest : std::min<int64_t>(ctas, int64_t(p.rest) * p.k_chunks));
  p.ctas = int(p.whole > 0 ? ctas : p.rest_ctas);
  return p;
}

// ---- the products on the tensor cores (gated_gemm.cu)

constexpr int kGatedPartT = 256;     // tokens of one MMA at most, half in each CTA
constexpr int kGatedMaxPairs = 80;   // most CTA pairs that splits are made for
constexpr int gated_tile_w(bool backward) { return backward ? 256 : 128; }   // outputs of a pair's tile

// Splits of a reduction: a step costs the decoding of its weights whatever the tokens, so few
// tiles with many steps are slow (dx of 100 tokens, 4000 x 2048: 8 tiles of 127 steps, 65 us).
// Eight steps a split at least, and none of fewer than 24 (333 tokens, 1032 x 1088: 22.4 against
// 21.9).

// dx fills the pairs that its tiles leave idle, if those are half or more.  It keeps to two
// thirds of the SMs, and leaves the others to dB and dA beside it, unless it is long itself, 20
// steps for every pair (100 tokens, 4000 x 2048, 8 tiles of 126 steps: 6 splits 39 us, 9 splits
// 45; 16 tokens, 4096 x 4096, 16 tiles of 130: 3 splits 46 us, 4 splits 42).
inline int gated_dx_splits(int64_t tiles, int steps, int sms) {
  if (steps < 24) return 1;
  const int64_t pairs = std::min(std::max(sms / 2, 1), kGatedMaxPairs);
  const int64_t most = steps * tiles < 20 * pairs ? ((sms + 2) / 3 + tiles / 2) / tiles : pairs;
  return int(std::max<int64_t>(1, std::min<int64_t>({most, pairs / tiles, steps / 8})));
}

// The forward takes what costs least by these measured parts, in ns: 460 a step, 1,000 a tile,
// 3,500 for the launch that adds the splits up, and their sums written and read at 5 TB/s
// (64 tokens, 1000 x 4096, 8 tiles: 35 us, with 8 splits 17; 11008 x 4096, 86 tiles on 74 pairs:
// 67 us, with 3 splits 55; 14336 x 4096, 112 tiles: 68 us, with 2 to 5 splits 67 to 72).
constexpr int kGatedMaxFwdSplits = 16;
constexpr size_t kGatedMaxFwdSums = size_t(40) << 20;
inline size_t gated_fwd_sums(int64_t splits, int64_t M, int64_t N) {
  return size_t(splits) * size_t(M) * size_t(2 * N) * sizeof(float);
}
struct GatedFwdSplits {
  int splits;
  int64_t ns;
};
inline GatedFwdSplits gated_fwd_splits(int64_t M, int64_t N, int64_t tiles, int steps, int sms) {
  const int64_t pairs = std::max(sms / 2, 1);
  GatedFwdSplits best{1, INT64_MAX};
  for (int s = 1; s <= kGatedMaxFwdSplits; ++s) {
    if (s > 1 && (steps < 24 || steps / s < 8 || gated_fwd_sums(s, M, N) > kGatedMaxFwdSums)) break;
    const int64_t sums = s > 1 ? 3500 + int64_t(2 * gated_fwd_sums(s, M, N) / 5000) : 0;
    const int64_t ns = plan_cdiv(tiles * s, pairs) * (plan_cdiv(steps, s) * 460 + 1000) + sums;
    if (ns < best.ns) best = GatedFwdSplits{s, ns};
  }
  return best;
}

// Steps of 64 of the reduction: one projection's and the adapters' (forward), or both's (dx).
inline int64_t gated_steps(bool backward, int64_t N, int64_t K, int r) {
  return (backward ? 2 * plan_cdiv(N, 64) : K / 64) + 2 * ((r + 63) / 64);
}

// Splits' sums, fp32: [split][M][K] or, forward, [split][M][2][N].  In dx more rows make more
// tiles and so fewer splits: the size is the largest of any number of rows up to M, so that a
// workspace for M serves fewer.
constexpr int kGatedAlwaysStream = 16, kGatedMayStream = 32;   // tokens, see gated_streams
inline size_t gated_split_bytes(bool backward, int64_t M, int64_t N, int64_t K, int r) {
  const int64_t steps = gated_steps(backward, N, K, r);
  if (steps < 24) return 0;
  if (!backward)
    return M <= kGatedAlwaysStream ? 0 : std::min(kGatedMaxFwdSums, gated_fwd_sums(std::min<int64_t>(kGatedMaxFwdSplits, steps / 8), M, N));
  const int64_t col_tiles = plan_cdiv(K, gated_tile_w(true));
  int64_t rows = 0;
  for (int64_t m_tiles = 1; (m_tiles - 1) * kGatedPartT < M && 2 * m_tiles * col_tiles <= kGatedMaxPairs; ++m_tiles)
    rows = std::max(rows, std::min(kGatedMaxPairs / (m_tiles * col_tiles), steps / 8) * std::min(M, m_tiles * kGatedPartT));
  return size_t(rows) * size_t(K) * sizeof(float);
}

struct GatedGemmPlan {
  int parts;                // MMAs of 256 tokens a tile
  int half_steps;           // steps of 64 of one projection: forward K / 64, backward ceil(N / 64)
  int main_steps;           // half_steps, or both projections' (backward)
  int ad_steps;             // ceil(r / 64), of one projection
  int col_tiles, row_tiles, tile_rows;
  int splits;               // of the reduction
  int64_t tiles;            // of all splits
  int pairs;                // of CTAs
};

inline GatedGemmPlan gated_gemm_plan(bool backward, int64_t M, int64_t N, int64_t K, int r, int sms) {
  GatedGemmPlan p{};
  const int64_t col_tiles = plan_cdiv(backward ? K : N, gated_tile_w(backward));
  // Two MMAs a decoded weight tile where there are more tokens than one MMA takes and
  // one-MMA tiles would need a second wave of CTA pairs (the expert GEMM's rule).
  p.parts = M > kGatedPartT && M / kGatedPartT * col_tiles > sms / 2 ? 2 : 1;
  p.half_steps = int(backward ? plan_cdiv(N, 64) : K / 64);
  p.main_steps = backward ? 2 * p.half_steps : p.half_steps;
  p.ad_steps = (r + 63) / 64;
  p.col_tiles = int(col_tiles);
  p.row_tiles = int(plan_cdiv(M, int64_t(p.parts) * kGatedPartT));
  const int64_t tiles256 = int64_t(p.row_tiles) * p.col_tiles;
  const int steps = int(gated_steps(backward, N, K, r));
  p.splits = p.parts == 2 ? 1 : backward ? gated_dx_splits(tiles256, steps, sms) : gated_fwd_splits(M, N, tiles256, steps, sms).splits;
  // Forward: CTA pairs left over take tiles of fewer tokens, whose MMAs and epilogue are shorter
  // (333 tokens, 1032 x 1088: 21.4 -> 17.0 us; 256, 512 x 512: 18.3 -> 12.4).  Beside dx, dB and
  // dA run on them (with smaller tiles the backward of 512 tokens, 1024 x 1024, took 39 us, not 32).
  const int64_t spare = backward ? 1 : sms / 2 / (tiles256 * p.splits);
  if (spare > 1) p.row_tiles = int(std::max<int64_t>(p.row_tiles, std::min(p.row_tiles * spare, plan_cdiv(M, 64))));
  p.tile_rows = int((plan_cdiv(M, p.row_tiles) + 31) & ~int64_t(31));   // pieces of 32 tokens are stored whole
  p.row_tiles = int(plan_cdiv(M, p.tile_rows));
  p.tiles = int64_t(p.row_tiles) * p.col_tiles * p.splits;
  p.pairs = int(std::min<int64_t>(p.tiles, std::max(sms / 2, 1)));
  return p;
}

// ---- between the two

// Few tokens: stream the weights (16 tokens a pass) instead of feeding the GEMM.  Up to 16 tokens
// always (graphs of calls over weights larger than L2, r = 16, us, this against the GEMM with 16
// tokens: 4096 x 4096 18.6 and 25.7, 2560 x 2560 16.3 and 18.3, 4096 x 512 10.9 and 11.6, 8192 x
// 1024 16.5 and 16.6, 28672 x 8192 109 and 221).  From 17 to 32, two passes, where tiles are whole
// or have CTAs of their own (24 tokens: 11008 x 4096 47 and 53, 1000 x 4096 15 and 17, 1024 x 1024
// 11 and 15, 5504 x 4096 28 and 32, 14336 x 4096 58 and 63); where shares straddle tiles, what
// takes less by measured parts, in ns: here 8,700 (start and T), 990 a unit, 2,700 for joins
// behind tiles of a CTA's own or 5,500 without; there the splits' cost and 6,000.  4096 x 4096 28.6
// and 25.9, 2752 x 4096 23.9 and 21.9, 2560 x 2560 21.9 and 18.4, 8192 x 2048 25.2 and 23.5, 17920 x
// 4096 72 and 66 go to the GEMM, 7168 x 4096 35 and 38, 13824 x 5120 69 and 74, 12032 x 4096 52 and
// 53 do not.  It is off by up to 6 % where the GEMM has about as many tiles as there are pairs
// (9216 outputs, K 2048, 4096, 5120: 27, 42, 49 and 29, 44, 51, to the GEMM).  Rows from 6144 on
// always stream: their codes come slower to the GEMM (3000 x 6144 29 and 34, 4096 x 6144 and x 8192
// 35 and 35, 41 and 42, 2752 x 8192 34 and 33).
//
// A rule without M in each range: a workspace for M serves fewer rows, and the backward makes T by
// the kernel that made it in the forward.
inline bool gated_streams(int64_t M, int64_t N, int64_t K, int r, int sms) {
  if (M <= kGatedAlwaysStream) return true;
  if (M > kGatedMayStream) return false;
  const GatedDecodePlan d = gated_decode_plan(kGatedMayStream, N, K, sms);
  const bool straddle = d.rest > 0 && d.rest_ctas < 2 * d.rest;
  if (!straddle || K >= 6144) return true;
  const int64_t units = int64_t(d.whole) * d.k_chunks * 990 + int64_t(d.rest) * d.k_chunks * 990 / d.rest_ctas;
  const GatedFwdSplits g = gated_fwd_splits(kGatedMayStream, N, plan_cdiv(N, gated_tile_w(false)), int(gated_steps(false, N, K, r)), sms);
  return 8700 + units + (d.whole > 0 ? 2700 : 5500) <= 6000 + g.ns;
}

}  // namespace nf4
