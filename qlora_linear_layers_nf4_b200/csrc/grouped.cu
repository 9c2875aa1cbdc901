// QLoRA linear of a stack of experts: the launches of a call.  Every launch is
// prepared (its tensor maps encoded) before the first is enqueued, so a call
// that fails on the host enqueues nothing.
#include "expert_decode.h"
#include "expert_gemm.h"
#include "expert_grad.h"
#include "expert_rank.h"
#include "kernels.h"
#include "nf4_common.cuh"

namespace nf4 {
namespace {

// One [M, r] scratch matrix, sized for fp32 so that the same workspace serves
// every compute dtype; U's three 16-bit terms share two.
size_t mr_bytes(int64_t M, int r) { return (size_t(M) * size_t(r) * 4 + 255) / 256 * 256; }

// Few rows per expert: stream the weights (16 rows a pass) instead of feeding
// the GEMM, which spends the same time on one row of an expert as on 256.
// Measured, this against the GEMM, us: 8 experts of 4096 x 4096 with 4, 16 and 24
// rows on average 44, 63 and 84 against 68 to 69; 64 experts of 1024 x 2048 with
// 16 and 24 rows 69 and 86 against 75.
bool use_decode(int64_t M, int64_t E) { return M <= 16 * E; }

// Rows x r up to which T takes one small CTA per element instead of the GEMM: whole
// calls on 8 experts of 4096 x 4096, r = 64, with 16, 32 and 64 rows 40.5, 44.3 and
// 54.5 us against 42.0, 44.6 and 51.2.
constexpr int64_t kSmallT = 2048;

}  // namespace

// fwd: [T] [the decode kernel's partials and counters]; bwd: [T] [U] [U]
size_t grouped_workspace_bytes(bool backward, int64_t M, int64_t N, int64_t K, int r) {
  (void)N;
  (void)K;
  if (M < 0 || r < 0) return 0;
  return backward ? 3 * mr_bytes(M, r) : mr_bytes(M, r) + decode_scratch_bytes();
}

cudaError_t launch_grouped_fwd(const GroupedArgs& g, int sms, cudaStream_t st, int* launches) {
  const LinearArgs& a = g.lin;
  if (a.f32) return launch_grouped_fwd_f32(g, st, launches);
  void* T = a.t_out ? a.t_out : a.ws + kWsHeader;
  cudaError_t e;
  ExpertDecode d;
  if (use_decode(a.M, g.E) && d.prepare(g, T, a.ws + kWsHeader + mr_bytes(a.M, a.r), sms)) {
    ExpertRank t;
    const bool small = a.M * a.r <= kSmallT;
    if (!small && !t.prepare(g, kRankT, T, nullptr, nullptr, sms)) return cudaErrorInvalidValue;
    if (small) {
      e = launch_expert_t_small(g, T, d.p.counters, st, launches);
    } else {
      t.p.zero = d.p.counters;
      t.p.zero_n = kDecodeMaxCtas;
      e = t.run(st, launches);
    }
    return e == cudaSuccess ? d.run(st, launches) : e;
  }
  ExpertRank t;
  ExpertGemm y;
  if (!t.prepare(g, kRankT, T, nullptr, nullptr, sms) || !y.prepare(g, false, T, sms)) return cudaErrorInvalidValue;
  e = t.run(st, launches);
  if (e == cudaSuccess) e = y.run(st, launches);
  return e;
}

cudaError_t launch_grouped_bwd(const GroupedArgs& g, int sms, cudaStream_t st, int* launches) {
  const LinearArgs& a = g.lin;
  if (a.f32) return launch_grouped_bwd_f32(g, st, launches);
  uint8_t* ws = a.ws + kWsHeader;
  const void* T = a.t_in ? a.t_in : ws;
  uint8_t* U[3];
  for (int i = 0; i < 3; ++i) U[i] = ws + mr_bytes(a.M, a.r) + size_t(i) * size_t(a.M) * size_t(a.r) * 2;   // r % 8 == 0: 16-byte aligned
  ExpertRank t, u;
  ExpertGrad grad;
  ExpertGemm dx;
  bool ok = a.t_in != nullptr || t.prepare(g, kRankT, ws, nullptr, nullptr, sms);
  ok = ok && u.prepare(g, kRankU, U[0], U[1], U[2], sms);
  ok = ok && grad.prepare(g, T, U[0], a.f16 ? 2 : 3, sms);
  ok = ok && (a.dx == nullptr || dx.prepare(g, true, U[0], sms));
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (a.t_in == nullptr) e = t.run(st, launches);
  if (e == cudaSuccess) e = u.run(st, launches);
  if (e == cudaSuccess && a.dx != nullptr) e = dx.run(st, launches);
  if (e == cudaSuccess) e = grad.run(st, launches);
  return e;
}

}  // namespace nf4
