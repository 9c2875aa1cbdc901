// Which form a call of the 8-bit floating point linear takes.  Host arithmetic alone (no CUDA),
// so that the tests can ask.
#pragma once

#include <algorithm>
#include <cstdint>

namespace nf4 {

constexpr int kFp8Block = 128;   // columns (and rows of a weight) that share a scale

// ---- few tokens: the weight streamed (fp8_small_kernel), sixteen of its rows a CTA at a time

constexpr int kFp8SmallRows = 16;
constexpr int64_t kFp8SmallMaxCodes = 96 * 1024;         // M * K
inline int64_t fp8_small_groups(int64_t N) { return (N + kFp8SmallRows - 1) / kFp8SmallRows; }
inline int64_t fp8_small_ctas(int64_t N, int sms) { return std::min<int64_t>(fp8_small_groups(N), 2 * int64_t(sms)); }

// Up to eight tokens (one MMA column group) the weight is streamed.  Measured, this against
// the tensor-core kernel with the same codes, us: 4096 x 4096 with 1 and 8 tokens 6.5 and 7.6
// against 8.5 and 9.0; 1024 x 8192 5.2 and 6.5 against 7.0; 11008 x 4096 12.1 and 13.0 against
// 13.5 and 14.0; 4096 x 11008 12.4 and 15.2 against 13.8.
inline bool fp8_streams(int64_t M, int64_t K) { return M <= 8 && M * K <= kFp8SmallMaxCodes; }
// Every CTA quantizes all tokens again: up to two tokens of 4096 that costs less than a
// launch (1, 2, 4 tokens: 8.6, 10.2, 13.3 us; with a launch of its own before 9.6 to 9.8).
inline bool fp8_quantizes_inside(int64_t M, int64_t K) { return M * K <= 8192; }

// ---- the product on the tensor cores (fp8_gemm.cu)

constexpr int kFp8MaxParts = 8;
struct Fp8GemmPlan {
  int tile_n;              // 256: pairs of CTAs, 256 x 256; else 128 x tile_n
  int parts;               // CTAs (a cluster) that share a tile's blocks along K; of 128 x tile_n
};

inline Fp8GemmPlan fp8_gemm_plan(int64_t M, int64_t N, int64_t K, int sms) {
  auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int64_t row_tiles = cdiv(M, 128), kb = cdiv(K, kFp8Block);
  Fp8GemmPlan p{256, 1};
  if (M <= 128 || cdiv(M, 256) * cdiv(N, 256) * 2 < sms) {
    // Pairs would leave SMs idle: of narrower tiles, and parts of their blocks, what takes least
    // by these measured times, in ns: 230, 275 or 350 a block of 32, 64 or 128 columns, 1,000 a
    // tile and 2,500 to join parts.  16 tokens through 4096 x 4096 take 8.9 us (128 columns, four
    // parts) against 10.7 with 32 columns, through 1024 x 8192 7.1 against 16.0; 64 through 11008 x
    // 4096 14.6 with 128 columns, 21.3 with 64; 333 through 1000 x 2064 7.8 with 32, 8.8 with 128.
    int64_t best = INT64_MAX;
    const int64_t block_ns[3] = {350, 275, 230};
    for (int w = 0; w < 3; ++w)
      for (int s = 1; s <= kFp8MaxParts && (s == 1 || kb / s >= 2); s *= 2) {
        const int64_t tiles = row_tiles * cdiv(N, 128 >> w);
        // a tile a CTA, all at once: GPCs hold whole clusters (16 of eight did not fit: 11.4 us
        // against 7.1 of 8)
        if (s > 1 && tiles * s > (s == 8 ? sms * 2 / 3 : sms * 7 / 8)) break;
        const int64_t cost = cdiv(tiles, sms) * (cdiv(kb, s) * block_ns[w] + 1000) + (s > 1 ? 2500 : 0);
        if (cost < best) {
          best = cost;
          p.tile_n = 128 >> w;
          p.parts = s;
        }
      }
  }
  return p;
}

}  // namespace nf4
