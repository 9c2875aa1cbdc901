// QLoRA linear of a stack of experts on the CUDA cores: the fp32 mode.
//
// For the rows m of expert e (rows sorted by expert):
//     y  = x W'_e^T + T B_e^T (+ bias_e),   T = s x A_e^T
//     U  = s dy B_e,  dB_e = dy^T T,  dA_e = U^T x,  dx = dy W'_e + U A_e
// One kernel does every product: C(i, j) = alpha * (sum over up to two
// segments of a(i, kk) b(j, kk)) (+ bias(j)), each operand a dense matrix in
// either major order or the NF4 weight decoded on load.  An operand's token
// index is either its i (row products: y, T, U, dx) or its kk (the gradients
// dA, dB, a sum over an expert's rows); everything else of an expert sits a
// fixed stride behind the expert before.  64 x 64 tile a CTA, 256 threads with
// 4 x 4 sums each in fp32, the reduction in slices of 32 through shared memory
// with the next slice's loads in flight.  Small calls are bound by the latency of a
// slice (load, barrier, sums): the backward of 301 rows, 4 experts of 512 x 512, takes
// 134 us, 143 with slices of 16.
#include <algorithm>

#include <cuda_runtime.h>

#include "grouped.cuh"
#include "kernels.h"
#include "nf4_common.cuh"

namespace nf4 {
namespace {

constexpr int kSTile = 64;
constexpr int kSK = 32;               // reduction per slice, loaded as two halves of 16
constexpr int kSHalf = 16;
constexpr int kSThreads = 256;
constexpr int kSRow = kSTile + 4;

struct SimtOperand {
  const float* p;        // null: the NF4 weight
  int64_t ld;            // elements between consecutive stored rows
  int kmajor;            // 1: (i, kk) at p[i * ld + kk]; 0: at p[kk * ld + i]
  int token;             // 1: i is a row of the batch, 2: kk is; 0: the operand is the expert's
  int64_t stride;        // token == 0: elements of one expert
  int64_t extent;        // token != 1: number of valid i
};

struct SimtSegment {
  SimtOperand a, b;
  int64_t kdim;          // reduction length (unused when kk is a token)
};

struct SimtParams {
  SimtSegment seg[2];
  int nseg;
  int by_rows;           // 1: i is a row of the batch; 0: C is per expert, kk is
  int64_t rows;          // by_rows == 0: rows of an expert's C
  int64_t cols;
  float* c;              // row-major [*, cols]
  float alpha;
  const float* bias;     // [E, cols] or null
  int col_tiles, row_tiles;
  int E, M;
  const int32_t* offsets;
  // the NF4 weight
  const uint8_t* codes;
  const float* absmax;
  const uint8_t* absmax_q;
  const float* absmax_scale;
  int dq;
  int bs_shift;
  uint32_t* status;
};

__global__ void __launch_bounds__(kSThreads) grouped_simt_kernel(const SimtParams p) {
  __shared__ float sa[2][kSK * kSRow];
  __shared__ float sb[2][kSK * kSRow];
  __shared__ float lut[16];
  __shared__ GroupTable groups;
  const int t = threadIdx.x;
  if (t < 16) lut[t] = level(t);
  if (t < 32) build_groups(&groups, p.offsets, p.E, p.M, kSTile, blockIdx.x == 0 ? p.status : nullptr);
  __syncthreads();

  int e;
  int64_t i0, i_end;
  const int64_t j0 = int64_t(blockIdx.x % p.col_tiles) * kSTile;
  const int64_t row_tile = blockIdx.x / p.col_tiles;
  if (p.by_rows) {
    if (row_tile >= groups.tiles[p.E]) return;
    e = expert_of_tile(&groups, p.E, int(row_tile));
    i0 = groups.start[e] + (row_tile - groups.tiles[e]) * kSTile;
    i_end = groups.start[e + 1];
  } else {
    e = int(row_tile / p.row_tiles);
    i0 = (row_tile % p.row_tiles) * kSTile;
    i_end = p.rows;
  }
  const int64_t tok0 = groups.start[e], tok1 = groups.start[e + 1];

  // Four elements of half an operand's slice per thread.  kmajor: i = first + t / 4,
  // kk = k0 + 4 (t % 4) ..; otherwise kk = k0 + t / 16, i = first + 4 (t % 16) ..
  auto load_half = [&](const SimtOperand& o, int64_t first, int64_t extent, int64_t k0, int64_t kend, float (&v)[4]) {
    const int64_t i = o.kmajor ? first + (t >> 2) : first + 4 * (t & 15);
    const int64_t kk = o.kmajor ? k0 + 4 * (t & 3) : k0 + (t >> 4);
    const int64_t base = (o.token ? 0 : int64_t(e) * o.stride) + (o.kmajor ? i * o.ld + kk : kk * o.ld + i);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool ok = o.kmajor ? (i < extent && kk + u < kend) : (kk < kend && i + u < extent);
      float f = 0.0f;
      if (ok) {
        const int64_t at = base + u;
        if (o.p == nullptr) {
          const uint32_t byte = p.codes[at >> 1];
          const int64_t blk = at >> p.bs_shift;
          const float scale = p.dq ? __fmul_rn(float(p.absmax_q[blk]), *p.absmax_scale) : p.absmax[blk];
          f = __fmul_rn(lut[(at & 1) ? (byte & 15u) : (byte >> 4)], scale);
        } else {
          f = __ldg(o.p + at);
        }
      }
      v[u] = f;
    }
  };
  auto load = [&](const SimtOperand& o, int64_t first, int64_t extent, int64_t k0, int64_t kend, float (&v)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) load_half(o, first, extent, k0 + h * kSHalf, kend, v[h]);
  };
  auto park = [&](const SimtOperand& o, float* s, const float (&v)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (o.kmajor) s[(h * kSHalf + 4 * (t & 3) + u) * kSRow + (t >> 2)] = v[h][u];
        else s[(h * kSHalf + (t >> 4)) * kSRow + 4 * (t & 15) + u] = v[h][u];
      }
  };

  const int ty = t >> 4, tx = t & 15;
  float acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = 0.0f;

  for (int g = 0; g < p.nseg; ++g) {
    const SimtSegment& sg = p.seg[g];
    const int64_t kbeg = p.by_rows ? 0 : tok0, kend = p.by_rows ? sg.kdim : tok1;
    const int64_t slices = (kend - kbeg + kSK - 1) / kSK;
    const int64_t a_end = sg.a.token == 1 ? i_end : sg.a.extent;
    float va[2][4], vb[2][4];
    if (slices > 0) {
      load(sg.a, i0, a_end, kbeg, kend, va);
      load(sg.b, j0, sg.b.extent, kbeg, kend, vb);
    }
    for (int64_t s = 0; s < slices; ++s) {
      const int cur = int(s & 1);
      park(sg.a, sa[cur], va);
      park(sg.b, sb[cur], vb);
      __syncthreads();
      if (s + 1 < slices) {
        load(sg.a, i0, a_end, kbeg + (s + 1) * kSK, kend, va);
        load(sg.b, j0, sg.b.extent, kbeg + (s + 1) * kSK, kend, vb);
      }
      float sum[4][4];   // of the slice: short sums added to the long one lose less
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) sum[a][b] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < kSK; ++kk) {
        const float4 a4 = *reinterpret_cast<const float4*>(&sa[cur][kk * kSRow + 4 * ty]);
        const float4 b4 = *reinterpret_cast<const float4*>(&sb[cur][kk * kSRow + 4 * tx]);
        const float ar[4] = {a4.x, a4.y, a4.z, a4.w}, br[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) sum[a][b] = fmaf(ar[a], br[b], sum[a][b]);
      }
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] += sum[a][b];
    }
    __syncthreads();
  }

#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int64_t i = i0 + 4 * ty + a;
    if (i >= i_end) continue;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int64_t j = j0 + 4 * tx + b;
      if (j >= p.cols) continue;
      float v = __fmul_rn(p.alpha, acc[a][b]);
      if (p.bias != nullptr) v = __fadd_rn(v, __ldg(p.bias + int64_t(e) * p.cols + j));
      p.c[((p.by_rows ? 0 : int64_t(e) * p.rows) + i) * p.cols + j] = v;
    }
  }
}

SimtOperand token_rows(const void* p, int64_t ld, bool kmajor, int token, int64_t extent) {
  SimtOperand o{};
  o.p = static_cast<const float*>(p);
  o.ld = ld;
  o.kmajor = kmajor;
  o.token = token;
  o.extent = extent;
  return o;
}
SimtOperand of_expert(const void* p, int64_t ld, bool kmajor, int64_t stride, int64_t extent) {
  SimtOperand o{};
  o.p = static_cast<const float*>(p);
  o.ld = ld;
  o.kmajor = kmajor;
  o.stride = stride;
  o.extent = extent;
  return o;
}

SimtParams common(const GroupedArgs& g) {
  const LinearArgs& a = g.lin;
  SimtParams p{};
  p.nseg = 1;
  p.alpha = 1.0f;
  p.E = g.E;
  p.M = int(a.M);
  p.offsets = g.offsets;
  p.codes = a.w->codes;
  p.absmax = a.w->absmax;
  p.absmax_q = a.w->absmax_q;
  p.absmax_scale = a.w->absmax_scale;
  p.dq = a.w->double_quant ? 1 : 0;
  p.bs_shift = log2_block(a.w->block_size);
  p.status = a.status;
  return p;
}

bool set_grid(SimtParams& p, int64_t* ctas) {
  const int64_t ct = (p.cols + kSTile - 1) / kSTile;
  const int64_t rt = p.by_rows ? max_row_tiles(p.M, p.E, kSTile)
                               : ((p.rows + kSTile - 1) / kSTile) * p.E;
  if (ct * rt > int64_t(0x7fffffff)) return false;
  p.col_tiles = int(ct);
  p.row_tiles = p.by_rows ? 0 : int((p.rows + kSTile - 1) / kSTile);
  *ctas = ct * rt;
  return true;
}

cudaError_t run(const SimtParams& p, int64_t ctas, int id, cudaStream_t st, int* launches) {
  NF4_PROF_BEGIN(st, id);
  grouped_simt_kernel<<<unsigned(ctas), kSThreads, 0, st>>>(p);
  NF4_PROF_END(st, id);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

struct Launch {
  SimtParams p;
  int64_t ctas;
  int id;
};

bool add(Launch* list, int* n, const SimtParams& p, int id) {
  Launch& l = list[*n];
  l.p = p;
  l.id = id;
  if (!set_grid(l.p, &l.ctas)) return false;
  ++*n;
  return true;
}

SimtParams product_T(const GroupedArgs& g, void* T) {
  const LinearArgs& a = g.lin;
  SimtParams p = common(g);
  p.by_rows = 1;
  p.seg[0].a = token_rows(a.x, a.K, true, 1, 0);
  p.seg[0].b = of_expert(a.A, a.K, true, int64_t(a.r) * a.K, a.r);
  p.seg[0].kdim = a.K;
  p.cols = a.r;
  p.c = static_cast<float*>(T);
  p.alpha = a.s;
  return p;
}

size_t mr_bytes(int64_t M, int r) { return (size_t(M) * size_t(r) * sizeof(float) + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_grouped_fwd_f32(const GroupedArgs& g, cudaStream_t st, int* launches) {
  const LinearArgs& a = g.lin;
  void* T = a.t_out ? a.t_out : a.ws + kWsHeader;
  Launch l[2];
  int n = 0;
  bool ok = add(l, &n, product_T(g, T), kKGroupedT);
  SimtParams p = common(g);
  p.by_rows = 1;
  p.nseg = 2;
  p.seg[0].a = token_rows(a.x, a.K, true, 1, 0);
  p.seg[0].b = of_expert(nullptr, a.K, true, a.N * a.K, a.N);
  p.seg[0].kdim = a.K;
  p.seg[1].a = token_rows(T, a.r, true, 1, 0);
  p.seg[1].b = of_expert(a.B, a.r, true, a.N * a.r, a.N);
  p.seg[1].kdim = a.r;
  p.cols = a.N;
  p.c = static_cast<float*>(a.y);
  p.bias = static_cast<const float*>(a.bias);
  ok = ok && add(l, &n, p, kKGroupedFwd);
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < n && e == cudaSuccess; ++i) e = run(l[i].p, l[i].ctas, l[i].id, st, launches);
  return e;
}

cudaError_t launch_grouped_bwd_f32(const GroupedArgs& g, cudaStream_t st, int* launches) {
  const LinearArgs& a = g.lin;
  uint8_t* ws = a.ws + kWsHeader;
  const void* T = a.t_in ? a.t_in : ws;
  float* U = reinterpret_cast<float*>(ws + mr_bytes(a.M, a.r));
  Launch l[5];
  int n = 0;
  bool ok = a.t_in != nullptr || add(l, &n, product_T(g, ws), kKGroupedT);
  {  // U = s dy B_e
    SimtParams p = common(g);
    p.by_rows = 1;
    p.seg[0].a = token_rows(a.dy, a.N, true, 1, 0);
    p.seg[0].b = of_expert(a.B, a.r, false, a.N * a.r, a.r);
    p.seg[0].kdim = a.N;
    p.cols = a.r;
    p.c = U;
    p.alpha = a.s;
    ok = ok && add(l, &n, p, kKGroupedU);
  }
  {  // dB_e = dy^T T
    SimtParams p = common(g);
    p.rows = a.N;
    p.seg[0].a = token_rows(a.dy, a.N, false, 2, a.N);
    p.seg[0].b = token_rows(T, a.r, false, 2, a.r);
    p.cols = a.r;
    p.c = a.dB;
    ok = ok && add(l, &n, p, kKGroupedDB);
  }
  {  // dA_e = U^T x
    SimtParams p = common(g);
    p.rows = a.r;
    p.seg[0].a = token_rows(U, a.r, false, 2, a.r);
    p.seg[0].b = token_rows(a.x, a.K, false, 2, a.K);
    p.cols = a.K;
    p.c = a.dA;
    ok = ok && add(l, &n, p, kKGroupedDA);
  }
  if (a.dx != nullptr) {  // dx = dy W'_e + U A_e
    SimtParams p = common(g);
    p.by_rows = 1;
    p.nseg = 2;
    p.seg[0].a = token_rows(a.dy, a.N, true, 1, 0);
    p.seg[0].b = of_expert(nullptr, a.K, false, a.N * a.K, a.K);
    p.seg[0].kdim = a.N;
    p.seg[1].a = token_rows(U, a.r, true, 1, 0);
    p.seg[1].b = of_expert(a.A, a.K, false, int64_t(a.r) * a.K, a.K);
    p.seg[1].kdim = a.r;
    p.cols = a.K;
    p.c = static_cast<float*>(a.dx);
    ok = ok && add(l, &n, p, kKGroupedDx);
  }
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < n && e == cudaSuccess; ++i) e = run(l[i].p, l[i].ctas, l[i].id, st, launches);
  return e;
}

}  // namespace nf4
