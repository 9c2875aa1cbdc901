// Gated feed-forward layer on the CUDA cores: the fp32 mode, where every product and sum is an
// fp32 operation.
//
// One kernel does every product of both projections z:
//     C_z(i, j) = alpha sum over up to four segments of a(i, kk) b(j, kk)
// with each operand a dense matrix in either major order or a projection's NF4 weight decoded
// on load; a second form keeps the sums of both projections and finishes h = act(g) u.
// T x T tiles (64, or 32 where those would leave SMs idle), 256 threads, the reduction in
// slices of 32 through shared memory with the loads of the next two slices in flight; a
// slice's products are summed by themselves before they are added to the others.  What a
// slice takes is the latency of few warps, so where there are few tiles a cluster of CTAs
// shares a tile's slices and sums its parts through distributed shared memory in their order:
// the backward of 301 rows, 512 x 512 and r = 8 went from 96 to 55 us, and to 45 with U and dB,
// and dA and dx, in one launch each.
#include <algorithm>

#include <cuda_runtime.h>

#include "gated.h"
#include "gated_act.cuh"
#include "nf4_common.cuh"
#include "tc_common.cuh"

namespace nf4 {
namespace {

constexpr int kSK = 32;
constexpr int kSThreads = 256;
constexpr int kSMaxCluster = 8;

// Element (i, kk).  Contiguous runs of four stay inside an operand: every row length is a
// multiple of eight.
struct SimtOperand {
  const float* p;        // null: the NF4 weight w
  int w;
  int64_t ld;            // elements between consecutive stored rows
  int kmajor;            // 1: (i, kk) at p[i * ld + kk]; 0: at p[kk * ld + i]
  int64_t extent;        // of i
  int64_t z_stride;      // elements to the other projection's matrix
  int z_w;               // 1: the other projection's weight is the other one
};

struct SimtSegment {
  SimtOperand a, b;
  int64_t kdim;
};

struct SimtWeight {
  const uint8_t* codes;
  const float* absmax;
  const uint8_t* absmax_q;
  const float* absmax_scale;
};

struct SimtParams {
  SimtSegment seg[4];
  int nseg;
  int64_t rows, cols;
  float* c;              // [z][rows][cols]
  float alpha;
  int col_tiles;
  SimtWeight w[2];
  int dq, bs_shift;
  // the gated form: seg[0], seg[1] of projection 0, 2 and 3 of projection 1
  const float* bias;     // [2][cols] or null
  float* pre;            // [2][rows][cols] or null
  int act;
};

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Two products in one launch, where neither reads the other's result: the first one's tiles,
// then the second one's.
struct SimtPair {
  SimtParams p[2];
  int tiles[2];          // of one z
  int blocks0;           // of the first, all z
};

template <int T, bool GATED>
__global__ void __launch_bounds__(kSThreads, 2) gated_simt_kernel(const __grid_constant__ SimtPair pair) {
  constexpr int kRow = T + 4;
  constexpr int kLoads = T * kSK / 4 / kSThreads;      // runs of four a thread, per operand and slice
  // A thread has 4 x 4 results, so that eight values read from shared memory feed 16 FMAs (2 x 2
  // were bound by those reads); the 32 x 32 tile's 64 threads are there four times, each with
  // a quarter of a slice, joined at the end.
  constexpr int kOwn = 4;
  constexpr int kSide = T / kOwn, kTeams = kSThreads / (kSide * kSide);
  __shared__ __align__(16) float sa[2][kSK * kRow];
  __shared__ __align__(16) float sb[2][kSK * kRow];
  __shared__ float lut[16];
  const int t = threadIdx.x;
  if (t < 16) lut[t] = level(t);
  __syncthreads();
  const int which = !GATED && int(blockIdx.x) >= pair.blocks0 ? 1 : 0;
  const SimtParams& p = pair.p[which];
  const int block = int(blockIdx.x) - (which ? pair.blocks0 : 0);
  const int z = block / pair.tiles[which], tile = block - z * pair.tiles[which];
  const int64_t j0 = int64_t(tile % p.col_tiles) * T, i0 = int64_t(tile / p.col_tiles) * T;

  // Run l of a slice.  kmajor: index = (t + 256 l) / 8, kk = 4 (t % 8) ..; else kk, then index.
  struct Runs {
    int64_t at[kLoads];    // element of the run in slice 0
    int64_t step;          // elements to the next slice
    int left[kLoads];      // slices that have the run
  };
  auto runs = [&](const SimtOperand& o, int64_t first, int64_t kend) {
    Runs r;
    r.step = o.kmajor ? kSK : kSK * o.ld;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int q = t + kSThreads * l;
      const int64_t i = first + (o.kmajor ? q / (kSK / 4) : 4 * (q % (T / 4)));
      const int64_t kk = o.kmajor ? 4 * (q % (kSK / 4)) : q / (T / 4);
      r.at[l] = o.kmajor ? i * o.ld + kk : kk * o.ld + i;
      r.left[l] = i < o.extent ? int((kend - kk + kSK - 1) / kSK) : 0;
    }
    return r;
  };
  auto load = [&](const SimtOperand& o, const Runs& r, int slice, float4 (&v)[kLoads]) {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      v[l] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (slice >= r.left[l]) continue;
      const int64_t at = r.at[l] + slice * r.step;
      if (o.p != nullptr) {
        v[l] = __ldg(reinterpret_cast<const float4*>(o.p + z * o.z_stride + at));
      } else {   // as it lies, decoded when it is parked: nothing waits for the load here
        const SimtWeight& w = p.w[o.w ^ (z & o.z_w)];
        const int64_t blk = at >> p.bs_shift;
        v[l].x = __uint_as_float(uint32_t(__ldg(reinterpret_cast<const uint16_t*>(w.codes + (at >> 1)))));
        v[l].y = p.dq ? __uint_as_float(uint32_t(__ldg(w.absmax_q + blk))) : __ldg(w.absmax + blk);
        v[l].w = 1.0f;   // there
      }
    }
  };
  const float s_g[2] = {p.dq ? __ldg(p.w[0].absmax_scale) : 0.0f, p.dq ? __ldg(p.w[1].absmax_scale) : 0.0f};
  auto park = [&](const SimtOperand& o, float* s, float4 (&v)[kLoads]) {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int q = t + kSThreads * l;
      if (o.p == nullptr && v[l].w != 0.0f) {
        const uint32_t two = __float_as_uint(v[l].x);
        const float c = p.dq ? __fmul_rn(float(__float_as_uint(v[l].y)), s_g[o.w ^ (z & o.z_w)]) : v[l].y;
        v[l] = make_float4(__fmul_rn(lut[(two >> 4) & 15u], c), __fmul_rn(lut[two & 15u], c),
                           __fmul_rn(lut[two >> 12], c), __fmul_rn(lut[(two >> 8) & 15u], c));
      }
      if (o.kmajor) {
        float* d = s + 4 * (q % (kSK / 4)) * kRow + q / (kSK / 4);
        d[0] = v[l].x;
        d[kRow] = v[l].y;
        d[2 * kRow] = v[l].z;
        d[3 * kRow] = v[l].w;
      } else {
        *reinterpret_cast<float4*>(s + q / (T / 4) * kRow + 4 * (q % (T / 4))) = v[l];
      }
    }
  };

  const int team = t / (kSide * kSide), ty = t % (kSide * kSide) / kSide, tx = t % kSide;
  constexpr int kSets = GATED ? 2 : 1;
  float acc[kSets][kOwn][kOwn];
#pragma unroll
  for (int g = 0; g < kSets; ++g)
#pragma unroll
    for (int a = 0; a < kOwn; ++a)
#pragma unroll
      for (int b = 0; b < kOwn; ++b) acc[g][a][b] = 0.0f;

  const int part = blockIdx.y, parts = gridDim.y;   // CTAs of a cluster share the slices
  int cur = 0;
  auto segment = [&](const SimtSegment& sg, float (&into)[kOwn][kOwn]) {
    const int64_t all = (sg.kdim + kSK - 1) / kSK;
    const int begin = int(all * part / parts), slices = int(all * (part + 1) / parts);
    if (begin == slices) return;
    const Runs ra = runs(sg.a, i0, sg.kdim), rb = runs(sg.b, j0, sg.kdim);
    float4 va[2][kLoads], vb[2][kLoads];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load(sg.a, ra, begin + h, va[h]);
      load(sg.b, rb, begin + h, vb[h]);
    }
    auto slice = [&](int s, float4 (&xa)[kLoads], float4 (&xb)[kLoads]) {
      park(sg.a, sa[cur], xa);
      park(sg.b, sb[cur], xb);
      __syncthreads();
      load(sg.a, ra, s + 2, xa);
      load(sg.b, rb, s + 2, xb);
      float sum[kOwn][kOwn];
#pragma unroll
      for (int a = 0; a < kOwn; ++a)
#pragma unroll
        for (int b = 0; b < kOwn; ++b) sum[a][b] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < kSK / kTeams; ++kk) {
        const int row = (team * (kSK / kTeams) + kk) * kRow;
        const float4 a4 = *reinterpret_cast<const float4*>(&sa[cur][row + kOwn * ty]);
        const float4 b4 = *reinterpret_cast<const float4*>(&sb[cur][row + kOwn * tx]);
        const float ar[kOwn] = {a4.x, a4.y, a4.z, a4.w}, br[kOwn] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int a = 0; a < kOwn; ++a)
#pragma unroll
          for (int b = 0; b < kOwn; ++b) sum[a][b] = fmaf(ar[a], br[b], sum[a][b]);
      }
#pragma unroll
      for (int a = 0; a < kOwn; ++a)
#pragma unroll
        for (int b = 0; b < kOwn; ++b) into[a][b] += sum[a][b];
      cur ^= 1;   // the barrier of the next slice separates its writes from these reads' buffer
    };
    for (int s = begin; s < slices; s += 2) {
      slice(s, va[0], vb[0]);
      if (s + 1 < slices) slice(s + 1, va[1], vb[1]);
    }
  };
  if (GATED) {
    segment(p.seg[0], acc[0]);
    segment(p.seg[1], acc[0]);
    segment(p.seg[2], acc[kSets - 1]);
    segment(p.seg[3], acc[kSets - 1]);
  } else {
    for (int g = 0; g < p.nseg; ++g) segment(p.seg[g], acc[0]);
  }

  auto finish = [&](int row, int col, const float (&v)[kSets]) {   // of the tile
    const int64_t i = i0 + row, j = j0 + col;
    if (i >= p.rows || j >= p.cols) return;
    const int64_t at = i * p.cols + j;
    if (GATED) {
      float g = v[0], u = v[kSets - 1];
      if (p.bias != nullptr) {
        g = __fadd_rn(g, __ldg(p.bias + j));
        u = __fadd_rn(u, __ldg(p.bias + p.cols + j));
      }
      if (p.pre != nullptr) {
        p.pre[at] = g;
        p.pre[p.rows * p.cols + at] = u;
      }
      p.c[at] = gated::act<false>(p.act, g) * u;
    } else {
      p.c[z * p.rows * p.cols + at] = __fmul_rn(p.alpha, v[0]);
    }
  };
  float* mine[2] = {&sa[0][0], &sb[0][0]};   // sums, from here on
  auto store_sums = [&]() {
#pragma unroll
    for (int g = 0; g < kSets; ++g)
#pragma unroll
      for (int a = 0; a < kOwn; ++a)
        *reinterpret_cast<float4*>(&mine[g][(kOwn * ty + a) * T + kOwn * tx]) =
            make_float4(acc[g][a][0], acc[g][a][1], acc[g][a][2], acc[g][a][3]);
  };
  __syncthreads();
#pragma unroll
  for (int m = 1; m < kTeams; ++m) {
    if (team == m) store_sums();
    __syncthreads();
    if (team == 0) {
#pragma unroll
      for (int g = 0; g < kSets; ++g)
#pragma unroll
        for (int a = 0; a < kOwn; ++a)
#pragma unroll
          for (int b = 0; b < kOwn; ++b) acc[g][a][b] += mine[g][(kOwn * ty + a) * T + kOwn * tx + b];
    }
    __syncthreads();
  }
  if (parts == 1) {
    if (team != 0) return;
#pragma unroll
    for (int a = 0; a < kOwn; ++a)
#pragma unroll
      for (int b = 0; b < kOwn; ++b) {
        float v[kSets];
#pragma unroll
        for (int g = 0; g < kSets; ++g) v[g] = acc[g][a][b];
        finish(kOwn * ty + a, kOwn * tx + b, v);
      }
    return;
  }
  if (team == 0) store_sums();
  tc::cluster_sync();
  for (int e = T * T * part / parts + t; e < T * T * (part + 1) / parts; e += kSThreads) {
    float v[kSets];
#pragma unroll
    for (int g = 0; g < kSets; ++g) {
      float one[kSMaxCluster];
#pragma unroll
      for (int c = 0; c < kSMaxCluster; ++c)   // all on their way before the first is needed
        one[c] = c < parts ? ld_shared_cluster(tc::mapa_shared(tc::smem_u32(mine[g] + e), uint32_t(c))) : 0.0f;
      v[g] = one[0];
#pragma unroll
      for (int c = 1; c < kSMaxCluster; ++c)
        if (c < parts) v[g] += one[c];
    }
    finish(e / T, e % T, v);
  }
  tc::cluster_sync();   // the sums stay until all have read them
}

// dg, du
__global__ void __launch_bounds__(kSThreads)
    gated_grad_f32_kernel(const float* __restrict__ dh, const float* __restrict__ pre, float* __restrict__ d, int64_t n, int act) {
  for (int64_t i = int64_t(blockIdx.x) * kSThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kSThreads) {
    const gated::ActGrad a = gated::act_grad<false>(act, pre[i]);
    const float v = dh[i];
    d[i] = v * pre[n + i] * a.d;
    d[n + i] = v * a.a;
  }
}

SimtOperand dense(const void* p, int64_t ld, bool kmajor, int64_t extent, int64_t z_stride) {
  return SimtOperand{static_cast<const float*>(p), 0, ld, kmajor ? 1 : 0, extent, z_stride, 0};
}
SimtOperand weight(int w, int64_t ld, bool kmajor, int64_t extent) { return SimtOperand{nullptr, w, ld, kmajor ? 1 : 0, extent, 0, 0}; }

SimtParams common(const GatedArgs& a) {
  SimtParams p{};
  p.alpha = 1.0f;
  for (int z = 0; z < 2; ++z) p.w[z] = SimtWeight{a.w[z]->codes, a.w[z]->absmax, a.w[z]->absmax_q, a.w[z]->absmax_scale};
  p.dq = a.w[0]->double_quant ? 1 : 0;
  p.bs_shift = log2_block(a.w[0]->block_size);
  p.act = a.act;
  return p;
}

struct Launch {
  SimtParams p;
  int zs, id;            // results (projections) of the launch
  bool gated;
};

int64_t slices_of(const Launch& l) {
  int64_t most = 0;
  for (int g = 0; g < (l.gated ? 4 : l.p.nseg); ++g) most = std::max(most, (l.p.seg[g].kdim + kSK - 1) / kSK);
  return most;
}
int64_t col_tiles(const Launch& l, int64_t t) { return (l.p.cols + t - 1) / t; }
int64_t tiles_of(const Launch& l, int64_t t) { return (l.p.rows + t - 1) / t * col_tiles(l, t); }

// Parts of a tile's slices: a power of two (clusters of seven waited for each other: 68 us
// against 55 for the backward of 301 rows, 512 x 512), such that all run at once at two CTAs
// an SM, an eighth of them left to the GPCs' remainders, and two slices a part at least.
int64_t parts_of(int64_t slices, int64_t tiles, int sms) {
  int64_t parts = 1;
  while (parts < kSMaxCluster && 2 * parts * tiles <= 2 * int64_t(sms) * 7 / 8 && slices >= 4 * parts) parts *= 2;
  return parts;
}

// The tiles are counted in 32 bits (those of both products of a launch together).
bool fits(const Launch& l) { return tiles_of(l, 32) * l.zs <= int64_t(0x3fffffff); }

// One product, or two that do not read each other's results.
cudaError_t run(const Launch& a, const Launch* b, int sms, cudaStream_t st, int* launches) {
  const Launch* l[2] = {&a, b};
  const int n = b != nullptr ? 2 : 1;
  int64_t blocks[2], slices = 0;
  auto count = [&](int64_t t) {   // CTAs of one part
    int64_t all = 0;
    for (int i = 0; i < n; ++i) all += blocks[i] = tiles_of(*l[i], t) * l[i]->zs;
    return all;
  };
  bool narrow = true;
  for (int i = 0; i < n; ++i) {
    slices = std::max(slices, slices_of(*l[i]));
    narrow = narrow && (l[i]->p.rows <= 32 || l[i]->p.cols <= 32);
  }
  // 64 x 64 tiles, which take half of the instructions a product, where their parts are enough
  // for the SMs.
  const int64_t wide = count(64);
  const bool large = !narrow && wide * parts_of(slices, wide, sms) >= sms;
  const int64_t t = large ? 64 : 32, all = count(t), parts = parts_of(slices, all, sms);
  SimtPair pair{};
  for (int i = 0; i < n; ++i) {
    pair.p[i] = l[i]->p;
    pair.p[i].col_tiles = int(col_tiles(*l[i], t));
    pair.tiles[i] = int(tiles_of(*l[i], t));
  }
  pair.blocks0 = int(blocks[0]);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(all), unsigned(parts), 1);
  cfg.blockDim = dim3(kSThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = unsigned(parts);
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  NF4_PROF_BEGIN(st, a.id);
  cudaError_t e;
  if (a.gated) e = large ? cudaLaunchKernelEx(&cfg, gated_simt_kernel<64, true>, pair) : cudaLaunchKernelEx(&cfg, gated_simt_kernel<32, true>, pair);
  else e = large ? cudaLaunchKernelEx(&cfg, gated_simt_kernel<64, false>, pair) : cudaLaunchKernelEx(&cfg, gated_simt_kernel<32, false>, pair);
  NF4_PROF_END(st, a.id);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

Launch product_T(const GatedArgs& a, void* T) {
  Launch l{common(a), 2, kKGatedT, false};
  l.p.nseg = 1;
  l.p.seg[0] = SimtSegment{dense(a.x, a.K, true, a.M, 0), dense(a.A, a.K, true, a.r, int64_t(a.r) * a.K), a.K};
  l.p.rows = a.M;
  l.p.cols = a.r;
  l.p.c = static_cast<float*>(T);
  l.p.alpha = a.s;
  return l;
}

size_t t_bytes(int64_t M, int r) { return (2 * size_t(M) * size_t(r) * 4 + 255) / 256 * 256; }

}  // namespace

// [T] and, backward, [U] [dg, du]
size_t gated_f32_workspace_bytes(bool backward, int64_t M, int64_t N, int r) {
  return backward ? 2 * t_bytes(M, r) + (2 * size_t(M) * size_t(N) * 4 + 255) / 256 * 256 : t_bytes(M, r);
}

cudaError_t launch_gated_fwd_f32(const GatedArgs& a, int sms, cudaStream_t st, int* launches) {
  float* T = a.t_out != nullptr ? static_cast<float*>(a.t_out) : reinterpret_cast<float*>(a.ws + kWsHeader);
  const Launch t = product_T(a, T);
  Launch h{common(a), 1, kKGatedFwd, true};
  for (int z = 0; z < 2; ++z) {
    h.p.seg[2 * z] = SimtSegment{dense(a.x, a.K, true, a.M, 0), weight(z, a.K, true, a.N), a.K};
    h.p.seg[2 * z + 1] = SimtSegment{dense(T + int64_t(z) * a.M * a.r, a.r, true, a.M, 0),
                                     dense(static_cast<const float*>(a.B) + int64_t(z) * a.N * a.r, a.r, true, a.N, 0), a.r};
  }
  h.p.rows = a.M;
  h.p.cols = a.N;
  h.p.c = static_cast<float*>(a.h);
  h.p.bias = static_cast<const float*>(a.bias);
  h.p.pre = static_cast<float*>(a.pre_out);
  if (!fits(t) || !fits(h)) return cudaErrorInvalidValue;
  const cudaError_t e = run(t, nullptr, sms, st, launches);
  return e == cudaSuccess ? run(h, nullptr, sms, st, launches) : e;
}

cudaError_t launch_gated_bwd_f32(const GatedArgs& a, int sms, cudaStream_t st, int* launches) {
  uint8_t* ws = a.ws + kWsHeader;
  float* U = reinterpret_cast<float*>(ws + t_bytes(a.M, a.r));
  float* d = reinterpret_cast<float*>(ws + 2 * t_bytes(a.M, a.r));
  const float* T = a.t_in != nullptr ? static_cast<const float*>(a.t_in) : reinterpret_cast<const float*>(ws);
  const int64_t mn = a.M * a.N, mr = a.M * a.r;
  const bool with_t = a.t_in == nullptr, with_dx = a.dx != nullptr;
  const Launch t = product_T(a, ws);
  Launch u{}, db{}, da{}, dx{};
  {  // U_z = s d_z B_z
    u = Launch{common(a), 2, kKGatedU, false};
    u.p.nseg = 1;
    u.p.seg[0] = SimtSegment{dense(d, a.N, true, a.M, mn), dense(a.B, a.r, false, a.r, a.N * a.r), a.N};
    u.p.rows = a.M;
    u.p.cols = a.r;
    u.p.c = U;
    u.p.alpha = a.s;
  }
  {  // dB_z = d_z^T T_z
    db = Launch{common(a), 2, kKGatedDB, false};
    db.p.nseg = 1;
    db.p.seg[0] = SimtSegment{dense(d, a.N, false, a.N, mn), dense(T, a.r, false, a.r, mr), a.M};
    db.p.rows = a.N;
    db.p.cols = a.r;
    db.p.c = a.dB;
  }
  {  // dA_z = U_z^T x
    da = Launch{common(a), 2, kKGatedDA, false};
    da.p.nseg = 1;
    da.p.seg[0] = SimtSegment{dense(U, a.r, false, a.r, mr), dense(a.x, a.K, false, a.K, 0), a.M};
    da.p.rows = a.r;
    da.p.cols = a.K;
    da.p.c = a.dA;
  }
  if (with_dx) {  // dx = sum_z d_z W'_z + U_z A_z
    dx = Launch{common(a), 1, kKGatedDx, false};
    dx.p.nseg = 4;
    for (int z = 0; z < 2; ++z) {
      dx.p.seg[z] = SimtSegment{dense(d + z * mn, a.N, true, a.M, 0), weight(z, a.K, false, a.K), a.N};
      dx.p.seg[2 + z] = SimtSegment{dense(U + z * mr, a.r, true, a.M, 0),
                                    dense(static_cast<const float*>(a.A) + int64_t(z) * a.r * a.K, a.K, false, a.K, 0), a.r};
    }
    dx.p.rows = a.M;
    dx.p.cols = a.K;
    dx.p.c = static_cast<float*>(a.dx);
  }
  if (!fits(t) || !fits(u) || !fits(db) || !fits(da) || (with_dx && !fits(dx))) return cudaErrorInvalidValue;
  NF4_PROF_BEGIN(st, kKGatedAct);
  gated_grad_f32_kernel<<<unsigned(std::max<int64_t>(1, std::min<int64_t>((mn + kSThreads - 1) / kSThreads, int64_t(sms) * 8))), kSThreads, 0, st>>>(
      static_cast<const float*>(a.dh), static_cast<const float*>(a.pre_in), d, mn, a.act);
  NF4_PROF_END(st, kKGatedAct);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  if (e == cudaSuccess && with_t) e = run(t, nullptr, sms, st, launches);
  if (e == cudaSuccess) e = run(u, &db, sms, st, launches);
  if (e == cudaSuccess) e = with_dx ? run(dx, &da, sms, st, launches) : run(da, nullptr, sms, st, launches);
  return e;
}

}  // namespace nf4
