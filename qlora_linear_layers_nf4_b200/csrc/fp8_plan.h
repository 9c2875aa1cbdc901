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

// Up to eight tokens (one MMA column group) the weight is streamed, where that takes less than the
// tensor-core kernel (codes given, graphs of calls over weights larger than L2, us, this against
// that):
//   1 and 8 tokens, 4096 x 4096 6.4 and 7.6 against 8.4 and 9.0; 11008 x 4096 11.9 and 12.6 against 13.5
//     and 13.4; 2048 x 2048 3.9 and 4.1 against 6.5 and 6.0; 1024 x 8192 6.9 and 8.1 against 7.9 and 8.0.
//   Many codes in shared memory cost it CTAs: 4096 x 11008 with 4 and 8 tokens 13.2 and 15.1
//     against 13.4 and 13.1, 4096 x 14336 with 3 and 6 15.5 and 17.5 against 15.5.
//   From more than a tile of 128 outputs an SM on the tensor-core kernel takes a second round:
//     28672 x 8192 with 1 and 8 tokens 40 and 44 against 47 and 49, 24576 x 14336 with 6 67 against 78.
//   Where it fills two thirds of the SMs or more with one round it is as fast or faster: 14336 x
//     4096 13.9 and 14.9 against 14.9 and 14.6, 16384 x 5120 21 and 23 against 18, 16384 x 11008 36 and 41
//     against 36 and 35.
//   Few outputs of long rows are shared by clusters there: 1024 x 14336 with 1 and 6 tokens 10.6 and
//     12.5 against 9.2 and 9.6, 2048 x 28672 with 3 20.2 against 18.5.
// Up to 11 % the other way are left: streamed, 8192 x 11008 with 4 tokens 23.1 against 20.9, 11008 x 5120
// with 8 16.3 against 15.5; not streamed, 11008 x 8192 with 6 22.7 against 21.9, 11008 x 28672 with 2 67
// against 60.
inline bool fp8_streams(int64_t M, int64_t N, int64_t K, int sms) {
  if (M > 8 || K > 8 * N) return false;
  const int64_t tiles = (N + 127) / 128;
  return tiles > sms ? M * K <= kFp8SmallMaxCodes : 3 * tiles <= 2 * int64_t(sms) && M * K <= 48 * 1024;
}
// Every CTA quantizes all tokens again, which costs less than a launch for few elements, and while
// the weight is not so long that its streaming waits (whole calls, us, inside against a launch of
// its own): 4096 x 4096 with 1 and 2 tokens 7.6 and 9.1 against 8.4 and 8.6, 2048 x 2048 with 1 and 4
// 4.4 and 6.0 against 6.2 and 6.7, 1024 x 8192 8.7 against 9.4; 8192 x 4096 12.0 against 12.6, 11008 x
// 4096 13.9 against 13.6 to 14.7, 14336 x 4096 17.3 against 16.4, 32000 x 2048 18.9 against 18.7.
inline bool fp8_quantizes_inside(int64_t M, int64_t N, int64_t K) {
  const int64_t weight = N * K, mega = int64_t(1) << 20;
  return weight <= 48 * mega && M * K <= (weight <= 8 * mega ? 8192 : 5632);
}

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
