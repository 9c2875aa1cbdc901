// Gated feed-forward layer: the launches of a call, and the fp32 mode.  Every launch of the
// 16-bit modes is prepared (its tensor maps encoded) before the first is enqueued, so a
// call that fails on the host enqueues nothing.
#include <algorithm>

#include "gated.h"
#include "gated_act.cuh"
#include "gated_decode.h"
#include "gated_rank.h"
#include "nf4_common.cuh"

namespace nf4 {
namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
size_t mr_bytes(int64_t M, int r, size_t size) { return align256(size_t(M) * size_t(r) * size); }
size_t pair_bytes(int64_t M, int64_t N, size_t size) { return align256(2 * size_t(M) * size_t(N) * size); }

// Few tokens: stream the weights (16 tokens a pass) instead of feeding the GEMM.
bool use_decode(int64_t M) { return M <= 32; }

// ------------------------------------------------------------------ fp32 mode
//
// The two linear layers and their backward by the dense layer's fp32 kernels, with the
// activation's products between: a reference mode.

constexpr int kElThreads = 256;

__global__ void __launch_bounds__(kElThreads) gated_act_f32_kernel(const float* __restrict__ pre, float* __restrict__ h,
                                                                   int64_t n, int act) {
  for (int64_t i = int64_t(blockIdx.x) * kElThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kElThreads)
    h[i] = gated::act<false>(act, pre[i]) * pre[n + i];
}

__global__ void __launch_bounds__(kElThreads)
    gated_grad_f32_kernel(const float* __restrict__ dh, const float* __restrict__ pre, float* __restrict__ d, int64_t n, int act) {
  for (int64_t i = int64_t(blockIdx.x) * kElThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kElThreads) {
    const gated::ActGrad a = gated::act_grad<false>(act, pre[i]);
    const float v = dh[i];
    d[i] = v * pre[n + i] * a.d;
    d[n + i] = v * a.a;
  }
}

__global__ void __launch_bounds__(kElThreads) gated_add_f32_kernel(float* __restrict__ to, const float* __restrict__ from, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * kElThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kElThreads) to[i] += from[i];
}

unsigned el_grid(int64_t n, int sms) {
  return unsigned(std::max<int64_t>(1, std::min<int64_t>((n + kElThreads - 1) / kElThreads, int64_t(sms) * 8)));
}

cudaError_t launched(cudaStream_t st, int id, int* launches) {
  NF4_PROF_END(st, id);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

// One projection's layer, as the dense fp32 kernels take it (T or U in ws).
LinearArgs f32_linear(const GatedArgs& a, int z) {
  LinearArgs l{};
  l.w = a.w[z];
  l.M = a.M;
  l.N = a.N;
  l.K = a.K;
  l.r = a.r;
  l.s = a.s;
  l.f32 = 1;
  l.x = a.x;
  l.A = static_cast<const float*>(a.A) + int64_t(z) * a.r * a.K;
  l.B = static_cast<const float*>(a.B) + int64_t(z) * a.N * a.r;
  l.ws = a.ws;
  l.status = a.status;
  return l;
}

cudaError_t fwd_f32(const GatedArgs& a, int sms, cudaStream_t st, int* launches) {
  const int64_t mn = a.M * a.N;
  float* pre = a.pre_out != nullptr ? static_cast<float*>(a.pre_out)
                                    : reinterpret_cast<float*>(a.ws + kWsHeader + linear_workspace_bytes(false, a.M, a.N, a.K, a.r));
  for (int z = 0; z < 2; ++z) {
    LinearArgs l = f32_linear(a, z);
    l.bias = a.bias != nullptr ? static_cast<const float*>(a.bias) + z * a.N : nullptr;
    l.y = pre + z * mn;
    l.t_out = a.t_out != nullptr ? static_cast<float*>(a.t_out) + int64_t(z) * a.M * a.r : nullptr;
    const cudaError_t e = launch_linear_fwd_f32(l, st, launches);
    if (e != cudaSuccess) return e;
  }
  NF4_PROF_BEGIN(st, kKGatedAct);
  gated_act_f32_kernel<<<el_grid(mn, sms), kElThreads, 0, st>>>(pre, static_cast<float*>(a.h), mn, a.act);
  return launched(st, kKGatedAct, launches);
}

cudaError_t bwd_f32(const GatedArgs& a, int sms, cudaStream_t st, int* launches) {
  const int64_t mn = a.M * a.N, mk = a.M * a.K;
  uint8_t* ws = a.ws + kWsHeader + linear_workspace_bytes(true, a.M, a.N, a.K, a.r);
  float* d = reinterpret_cast<float*>(ws);
  float* dx1 = reinterpret_cast<float*>(ws + pair_bytes(a.M, a.N, 4));
  NF4_PROF_BEGIN(st, kKGatedAct);
  gated_grad_f32_kernel<<<el_grid(mn, sms), kElThreads, 0, st>>>(static_cast<const float*>(a.dh),
                                                                 static_cast<const float*>(a.pre_in), d, mn, a.act);
  cudaError_t e = launched(st, kKGatedAct, launches);
  for (int z = 0; z < 2 && e == cudaSuccess; ++z) {
    LinearArgs l = f32_linear(a, z);
    l.dy = d + z * mn;
    l.t_in = a.t_in != nullptr ? static_cast<const float*>(a.t_in) + int64_t(z) * a.M * a.r : nullptr;
    l.dA = a.dA + int64_t(z) * a.r * a.K;
    l.dB = a.dB + int64_t(z) * a.N * a.r;
    l.dx = a.dx == nullptr ? nullptr : z == 0 ? a.dx : dx1;
    e = launch_linear_bwd_f32(l, st, launches);
  }
  if (e != cudaSuccess || a.dx == nullptr) return e;
  NF4_PROF_BEGIN(st, kKGatedAct);
  gated_add_f32_kernel<<<el_grid(mk, sms), kElThreads, 0, st>>>(static_cast<float*>(a.dx), dx1, mk);
  return launched(st, kKGatedAct, launches);
}

}  // namespace

// 16-bit: fwd [T] [the decode kernel's partials and counters]; bwd [T] [terms of U] [dg, du].
// fp32: the dense layer's, then fwd [g, u]; bwd [dg, du] [the second projection's dx].
size_t gated_workspace_bytes(bool backward, bool f32, int64_t M, int64_t N, int64_t K, int r) {
  if (M < 0 || N < 0 || K < 0 || r < 0) return 0;
  if (f32)
    return linear_workspace_bytes(backward, M, N, K, r) + pair_bytes(M, N, 4) + (backward ? align256(size_t(M) * size_t(K) * 4) : 0);
  const size_t t = mr_bytes(2 * M, r, 2);
  return backward ? t + mr_bytes(6 * M, r, 2) + pair_bytes(M, N, 2) : t + gated_decode_scratch_bytes();
}

cudaError_t launch_gated_fwd(const GatedArgs& a, int sms, cudaStream_t st, int* launches) {
  if (a.f32) return fwd_f32(a, sms, st, launches);
  void* T = a.t_out != nullptr ? a.t_out : a.ws + kWsHeader;
  GatedDecode d;
  if (use_decode(a.M)) {
    if (!d.prepare(a, T, a.ws + kWsHeader + mr_bytes(2 * a.M, a.r, 2), sms)) return cudaErrorInvalidValue;
    const cudaError_t e = launch_gated_t_small(a, T, d.p.counters, st, launches);
    return e == cudaSuccess ? d.run(st, launches) : e;
  }
  GatedRank t;
  GatedGemm h;
  if (!t.prepare(a, kGatedT, nullptr, nullptr, T, sms) || !h.prepare(a, false, a.x, T, sms)) return cudaErrorInvalidValue;
  const cudaError_t e = t.run(st, launches);
  return e == cudaSuccess ? h.run(st, launches) : e;
}

cudaError_t launch_gated_bwd(const GatedArgs& a, int sms, cudaStream_t st, int* launches) {
  if (a.f32) return bwd_f32(a, sms, st, launches);
  uint8_t* ws = a.ws + kWsHeader;
  uint8_t* U = ws + mr_bytes(2 * a.M, a.r, 2);
  uint8_t* d = U + mr_bytes(6 * a.M, a.r, 2);
  const void* T = a.t_in != nullptr ? a.t_in : ws;
  GatedRank t, u, db, da;
  GatedGemm dx;
  // T again comes from the kernel that made it in the forward: the same bits
  const bool small_t = use_decode(a.M);
  bool ok = a.t_in != nullptr || small_t || t.prepare(a, kGatedT, nullptr, nullptr, ws, sms);
  ok = ok && u.prepare(a, kGatedU, nullptr, d, U, sms);
  ok = ok && db.prepare(a, kGatedDB, T, nullptr, a.dB, sms);
  ok = ok && da.prepare(a, kGatedDA, U, nullptr, a.dA, sms);
  ok = ok && (a.dx == nullptr || dx.prepare(a, true, d, U, sms));
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (a.t_in == nullptr) e = small_t ? launch_gated_t_small(a, ws, nullptr, st, launches) : t.run(st, launches);
  if (e == cudaSuccess) e = u.run(st, launches);
  if (e == cudaSuccess && a.dx != nullptr) e = dx.run(st, launches);
  if (e == cudaSuccess) e = db.run(st, launches);
  if (e == cudaSuccess) e = da.run(st, launches);
  return e;
}

}  // namespace nf4
