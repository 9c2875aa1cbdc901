// Host interface of the gated layer's rank-r products (gated_rank.cu).
#pragma once

#include <cuda.h>

#include "gated.h"

namespace nf4 {

enum GatedRankKind {
  kGatedT = 0,   // T_p = s x A_p^T                        (tiles of tokens, reduction over K)
  kGatedDA,      // dA_p = U_p^T x                         (tiles of K, reduction over tokens)
  kGatedU,       // U_p = s d_p B_p, and d_p itself        (tiles of tokens, reduction over N)
  kGatedDB       // dB_p = d_p^T T_p                       (tiles of N, reduction over tokens)
};

struct GatedRankParams {
  int M, N, K, r;
  int red_steps;       // steps of 64 of the reduction
  int slices;          // CTAs of a cluster, which share a tile's reduction
  int f16, act;
  int terms;           // 16-bit terms that hold a d or a U
  float scale;         // s
  const uint16_t* dh;  // [M][N]
  const uint16_t* pre; // [2][M][N]
  uint16_t* d;         // kGatedU: dg, du [2][M][N], rounded
  uint16_t* out16;     // T [2][M][r] or the terms of U [2][terms][M][r]
  float* out32;        // dA [2][r][K] or dB [2][N][r]
  uint32_t* status;
};

// One product, prepared on the host before the first launch of a call.
struct GatedRank {
  GatedRankKind kind;
  CUtensorMap ma, mb;
  GatedRankParams p;
  dim3 grid;
  bool prepare(const GatedArgs& a, GatedRankKind kind, const void* in, void* d, void* out, int sms);
  cudaError_t run(cudaStream_t st, int* launches, bool beside = false) const;
};

constexpr int gated_terms(bool f16) { return f16 ? 2 : 3; }

}  // namespace nf4
