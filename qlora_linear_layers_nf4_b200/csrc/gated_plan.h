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
inline int gated_fwd_splits(int64_t M, int64_t N, int64_t tiles, int steps, int sms) {
  if (steps < 24) return 1;
  const int64_t pairs = std::max(sms / 2, 1);
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= kGatedMaxFwdSplits && (s == 1 || (steps / s >= 8 && gated_fwd_sums(s, M, N) <= kGatedMaxFwdSums)); ++s) {
    const int64_t sums = s > 1 ? 3500 + int64_t(2 * gated_fwd_sums(s, M, N) / 5000) : 0;
    const int64_t cost = plan_cdiv(tiles * s, pairs) * (plan_cdiv(steps, s) * 460 + 1000) + sums;
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// Splits' sums, fp32: [split][M][K] or, forward, [split][M][2][N].  In dx more rows make more
// tiles and so fewer splits: the size is the largest of any number of rows up to M, so that a
// workspace for M serves fewer.
inline size_t gated_split_bytes(bool backward, int64_t M, int64_t N, int64_t K) {
  if (!backward) return std::min(kGatedMaxFwdSums, gated_fwd_sums(kGatedMaxFwdSplits, M, N));
  const int64_t col_tiles = plan_cdiv(K, gated_tile_w(true));
  int64_t rows = 0;
  for (int64_t m_tiles = 1; (m_tiles - 1) * kGatedPartT < M && 2 * m_tiles * col_tiles <= kGatedMaxPairs; ++m_tiles)
    rows = std::max(rows, kGatedMaxPairs / (m_tiles * col_tiles) * std::min(M, m_tiles * kGatedPartT));
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
  const int steps = p.main_steps + 2 * p.ad_steps;
  p.splits = p.parts == 2 ? 1 : backward ? gated_dx_splits(tiles256, steps, sms) : gated_fwd_splits(M, N, tiles256, steps, sms);
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

// Few tokens: stream the weights (16 tokens a pass) instead of feeding the GEMM.  Measured, this
// against the GEMM, us: 11008 x 4096 with 1, 16, 17 and 32 tokens 27, 33, 51 and 52 against 53 to
// 58; 4096 x 4096 with 16 and 32 18 and 28 against 24 and 25; 1000 x 4096 with 1 and 32 10.6 and
// 15.1 against 16.5; 4096 x 1024 with 16 12.3 against 15.1.
inline bool gated_streams(int64_t M) { return M <= 32; }

}  // namespace nf4
