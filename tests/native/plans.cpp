// Answers which form a call takes, from the rules that the library is built with: a query a line on
// standard input, its fields a line on standard output.
#include <cstdio>

#include "fp8_plan.h"
#include "gated_plan.h"

int main() {
  char line[256], what[32];
  long long v[6];
  while (std::fgets(line, sizeof line, stdin)) {
    const int n = std::sscanf(line, "%31s %lld %lld %lld %lld %lld %lld", what, v, v + 1, v + 2, v + 3, v + 4, v + 5) - 1;
    const char w = what[0];
    if (w == 'd' && n == 4) {          // decode M N K sms
      const nf4::GatedDecodePlan p = nf4::gated_decode_plan(v[0], v[1], v[2], int(v[3]));
      std::printf("np %d row_tiles %d n_tiles %d k_chunks %d whole %d rest %d rest_ctas %d ctas %d\n", p.np, p.row_tiles,
                  p.n_tiles, p.k_chunks, p.whole, p.rest, p.rest_ctas, p.ctas);
    } else if (w == 'g' && n == 6) {   // gemm backward M N K r sms
      const nf4::GatedGemmPlan p = nf4::gated_gemm_plan(v[0] != 0, v[1], v[2], v[3], int(v[4]), int(v[5]));
      std::printf("parts %d main_steps %d ad_steps %d col_tiles %d row_tiles %d tile_rows %d splits %d tiles %lld pairs %d\n",
                  p.parts, p.main_steps, p.ad_steps, p.col_tiles, p.row_tiles, p.tile_rows, p.splits, (long long)p.tiles, p.pairs);
    } else if (w == 's' && n == 5) {   // streams M N K r sms
      std::printf("streams %d\n", nf4::gated_streams(v[0], v[1], v[2], int(v[3]), int(v[4])) ? 1 : 0);
    } else if (w == 'b' && n == 5) {   // bytes backward M N K r: of the splits' sums
      std::printf("bytes %zu\n", nf4::gated_split_bytes(v[0] != 0, v[1], v[2], v[3], int(v[4])));
    } else if (w == 'f' && n == 4) {   // fp8 M N K sms
      const nf4::Fp8GemmPlan p = nf4::fp8_gemm_plan(v[0], v[1], v[2], int(v[3]));
      std::printf("streams %d inside %d groups %lld ctas %lld tile_n %d parts %d\n", nf4::fp8_streams(v[0], v[1], v[2], int(v[3])) ? 1 : 0,
                  nf4::fp8_quantizes_inside(v[0], v[1], v[2]) ? 1 : 0, (long long)nf4::fp8_small_groups(v[1]),
                  (long long)nf4::fp8_small_ctas(v[1], int(v[3])), p.tile_n, p.parts);
    } else {
      std::fprintf(stderr, "unknown: %s", line);
      return 1;
    }
  }
  return 0;
}
