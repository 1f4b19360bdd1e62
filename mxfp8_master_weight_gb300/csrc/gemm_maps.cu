// TMA descriptors of a product's operands and scales.
#include "gemm_maps.h"

#include "gemm_impl.cuh"
#include "gemm_realign.cuh"

namespace mxfp8 {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library does not link the driver).
EncodeTiled encoder() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(p) : nullptr;
  }();
  return f;
}

cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle, const char** what) {
  const EncodeTiled f = encoder();
  if (f == nullptr) {
    *what = "gemm: cuTensorMapEncodeTiled is not available";
    return cudaErrorNotSupported;
  }
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult r = f(map, type, cuuint32_t(rank), const_cast<void*>(base), dims, strides, box, ones,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    *what = "gemm: TMA descriptor";
    return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

}  // namespace

static cudaError_t codes_map(const GemmOperand& o, int64_t k, int bytes, int rows, CUtensorMapSwizzle swizzle,
                             CUtensorMap* map, const char** what) {
  const cuuint64_t dims[2] = {cuuint64_t(o.colwise ? o.mn : k), cuuint64_t(o.colwise ? k : o.mn)};
  const cuuint64_t strides[1] = {cuuint64_t(o.ld)};
  const cuuint32_t box[2] = {cuuint32_t(bytes), cuuint32_t(rows)};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, o.codes, dims, strides, box, swizzle, what);
}

cudaError_t operand_map(const GemmOperand& o, int64_t k, int rows, CUtensorMap* map, const char** what) {
  return codes_map(o, k, 128, rows, CU_TENSOR_MAP_SWIZZLE_128B, map, what);
}

cudaError_t half_operand_map(const GemmOperand& o, int64_t k, CUtensorMap* map, const char** what) {
  return o.colwise ? codes_map(o, k, 64, 128, CU_TENSOR_MAP_SWIZZLE_64B, map, what)
                   : codes_map(o, k, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B, map, what);
}

cudaError_t residue_maps(const GemmOperand& o, int64_t k, CUtensorMap* maps, const char** what) {
  const int64_t rows = o.colwise ? k : o.mn, cols = o.colwise ? o.mn : k;
  const cuuint64_t strides[1] = {cuuint64_t(16 * o.ld)};
  const cuuint32_t box[2] = {kRawRow, 8};
  for (int s = 0; s < kResidues; ++s) {
    // a residue without rows takes row 0's bytes; its boxes land in rows that the matrix has not
    const uintptr_t first = reinterpret_cast<uintptr_t>(o.codes) + (s < rows ? s * o.ld : 0);
    const cuuint64_t dims[2] = {cuuint64_t(first % 16 + cols), cuuint64_t(s < rows ? (rows - s + 15) / 16 : 1)};
    const cudaError_t e = encode(&maps[s], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, reinterpret_cast<const void*>(first / 16 * 16),
                                 dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE, what);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t scale_map(const GemmOperand& o, int64_t k, int row_tiles, CUtensorMap* map, const char** what) {
  const int64_t along_k = scale_tiles_along_k(k, o.block);
  const cuuint64_t dims[3] = {kScaleTile / 4, cuuint64_t(along_k), cuuint64_t((o.mn + 127) / 128)};
  const cuuint64_t strides[2] = {kScaleTile, cuuint64_t(along_k * kScaleTile)};
  const cuuint32_t box[3] = {kScaleTile / 4, 1, cuuint32_t(row_tiles)};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, o.scale, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE, what);
}

}  // namespace mxfp8
