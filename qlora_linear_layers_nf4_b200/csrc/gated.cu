// Gated feed-forward layer: the launches of a call.  Every launch is prepared (its tensor maps
// encoded) before the first is enqueued, so a call that fails on the host enqueues nothing.

#include <algorithm>

#include "gated.h"
#include "gated_decode.h"
#include "gated_rank.h"
#include "nf4_common.cuh"

namespace nf4 {
namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
size_t mr_bytes(int64_t M, int r, size_t size) { return align256(size_t(M) * size_t(r) * size); }
size_t pair_bytes(int64_t M, int64_t N, size_t size) { return align256(2 * size_t(M) * size_t(N) * size); }

}  // namespace

// fwd [T] [the decode kernel's partials and counters]; bwd [T] [terms of U] [dg, du] [dx in splits]
size_t gated_workspace_bytes(bool backward, bool f32, int64_t M, int64_t N, int64_t K, int r) {
  if (M < 0 || N < 0 || K < 0 || r < 0) return 0;
  if (f32) return gated_f32_workspace_bytes(backward, M, N, r);
  const size_t t = mr_bytes(2 * M, r, 2);
  const size_t splits = gated_split_bytes(backward, M, N, K, r);
  return backward ? t + mr_bytes(6 * M, r, 2) + pair_bytes(M, N, 2) + splits : t + std::max(splits, gated_decode_scratch_bytes());
}

cudaError_t launch_gated_fwd(const GatedArgs& a, int sms, cudaStream_t st, int* launches) {
  if (a.f32) return launch_gated_fwd_f32(a, sms, st, launches);
  void* T = a.t_out != nullptr ? a.t_out : a.ws + kWsHeader;
  GatedDecode d;
  uint8_t* scratch = a.ws + kWsHeader + mr_bytes(2 * a.M, a.r, 2);
  if (gated_streams(a.M, a.N, a.K, a.r, sms)) {
    if (!d.prepare(a, T, scratch, sms)) return cudaErrorInvalidValue;
    const cudaError_t e = launch_gated_t_small(a, T, d.p.counters, st, launches);
    return e == cudaSuccess ? d.run(st, launches) : e;
  }
  GatedRank t;
  GatedGemm h;
  if (!t.prepare(a, kGatedT, nullptr, nullptr, T, sms) || !h.prepare(a, false, a.x, T, scratch, sms)) return cudaErrorInvalidValue;
  cudaError_t e = t.run(st, launches);
  if (e == cudaSuccess) e = h.run(st, launches);
  return e == cudaSuccess ? h.sum(st, launches) : e;
}

cudaError_t launch_gated_bwd(const GatedArgs& a, int sms, cudaStream_t st, int* launches) {
  if (a.f32) return launch_gated_bwd_f32(a, sms, st, launches);
  uint8_t* ws = a.ws + kWsHeader;
  uint8_t* U = ws + mr_bytes(2 * a.M, a.r, 2);
  uint8_t* d = U + mr_bytes(6 * a.M, a.r, 2);
  uint8_t* splits = d + pair_bytes(a.M, a.N, 2);
  const void* T = a.t_in != nullptr ? a.t_in : ws;
  GatedRank t, u, db, da;
  GatedGemm dx;
  // T again comes from the kernel that made it in the forward: the same bits
  const bool small_t = gated_streams(a.M, a.N, a.K, a.r, sms);
  bool ok = a.t_in != nullptr || small_t || t.prepare(a, kGatedT, nullptr, nullptr, ws, sms);
  ok = ok && u.prepare(a, kGatedU, nullptr, d, U, sms);
  ok = ok && db.prepare(a, kGatedDB, T, nullptr, a.dB, sms);
  ok = ok && da.prepare(a, kGatedDA, U, nullptr, a.dA, sms);
  ok = ok && (a.dx == nullptr || dx.prepare(a, true, d, U, splits, sms));
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (a.t_in == nullptr) e = small_t ? launch_gated_t_small(a, ws, nullptr, st, launches) : t.run(st, launches);
  if (e == cudaSuccess) e = u.run(st, launches);
  if (e == cudaSuccess && a.dx != nullptr) e = dx.run(st, launches);
  // dx lets dB start when U is complete, dB lets dA
  if (e == cudaSuccess) e = db.run(st, launches, /*beside=*/a.dx != nullptr);
  if (e == cudaSuccess) e = da.run(st, launches, /*beside=*/true);
  if (e == cudaSuccess && a.dx != nullptr) e = dx.sum(st, launches);
  return e;
}

}  // namespace nf4
