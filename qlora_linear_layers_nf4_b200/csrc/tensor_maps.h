// Host side: the driver's tensor map encoder, and TMA tensor maps of any rank up to 3
// (expert and 8-bit GEMMs).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace nf4 {

// cuTensorMapEncodeTiled.  It wants a current context, and a host thread that has
// launched nothing yet has none: there the device's context is made current, as the
// runtime does at a thread's first launch.
inline CUresult encode_tiled(CUtensorMap* map, CUtensorMapDataType type, cuuint32_t rank, void* base,
                             const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                             const cuuint32_t* elem_strides, CUtensorMapInterleave interleave,
                             CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion, CUtensorMapFloatOOBfill fill) {
  static const auto fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(p) : nullptr;
  }();
  if (fn == nullptr) return CUDA_ERROR_NOT_FOUND;
  CUresult r = fn(map, type, rank, base, dims, strides, box, elem_strides, interleave, swizzle, promotion, fill);
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess)
      r = fn(map, type, rank, base, dims, strides, box, elem_strides, interleave, swizzle, promotion, fill);
  }
  return r;
}

enum class MapElem { kU8, k16 };   // 1-byte or 2-byte elements

// Row-major tensor of `rank` dims, innermost first; strides of dims 1 .. in
// bytes (multiples of 16); box per dim.  What a box reads outside the tensor
// is zero.  False if it cannot be encoded.
inline bool encode_map(CUtensorMap* map, const void* base, MapElem elem, int rank, const uint64_t* dims,
                       const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle) {
  cuuint64_t d[3], s[2];
  cuuint32_t b[3], one[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i + 1 < rank) s[i] = strides[i];
  }
  return encode_tiled(map, elem == MapElem::kU8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                      cuuint32_t(rank), const_cast<void*>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool encode_map_2d(CUtensorMap* map, const void* base, MapElem elem, uint64_t inner, uint64_t outer,
                          uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
  const uint64_t dims[2] = {inner, outer}, strides[1] = {inner * (elem == MapElem::kU8 ? 1 : 2)};
  const uint32_t box[2] = {box_inner, box_outer};
  return encode_map(map, base, elem, 2, dims, strides, box, swizzle);
}

// A stack of `depth` matrices [outer][inner], densely packed: reads past the
// end of one matrix give zeros, not the next matrix.
inline bool encode_map_stack(CUtensorMap* map, const void* base, MapElem elem, uint64_t inner, uint64_t outer,
                             uint64_t depth, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
  const uint64_t row = inner * (elem == MapElem::kU8 ? 1 : 2);
  const uint64_t dims[3] = {inner, outer, depth}, strides[2] = {row, row * outer};
  const uint32_t box[3] = {box_inner, box_outer, 1};
  return encode_map(map, base, elem, 3, dims, strides, box, swizzle);
}

}  // namespace nf4
