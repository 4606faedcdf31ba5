// Host-side construction of TMA tensor maps (bf16, 2-D, 128-byte swizzle).
//
// The driver's cuTensorMapEncodeTiled is reached through the runtime's
// driver-entry-point query, so the library has no link-time dependency on
// libcuda and can be loaded (for argument validation and symbol checks) on a
// machine without a GPU driver.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace h3 {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  // looked up once per process (a function-local static: thread-safe initialisation)
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return PFN_cuTensorMapEncodeTiled_v12000(nullptr);
  }();
  return fn;
}

// The encoder is a driver call and wants a current context, which a host thread that has
// made no runtime call yet does not have: cudaSetDevice gives it the device's.
template <class... Args>
bool encode_tmap(Args... args) {
  const auto enc = tmap_encoder();
  if (!enc) return false;
  CUresult r = enc(args...);
  int dev = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess &&
      cudaSetDevice(dev) == cudaSuccess)
    r = enc(args...);
  return r == CUDA_SUCCESS;
}

// A row-major bf16 matrix [rows][cols] with a row pitch of `row_stride_elems`
// elements, read in boxes of box_rows x box_cols (box_cols * 2 must be 128 for
// the 128-byte swizzle).  Rows past `rows` read as zero.
inline bool make_tmap_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                              uint64_t row_stride_elems, uint32_t box_rows, uint32_t box_cols) {
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_stride_elems * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The same matrix in boxes of box_rows x 32 elements (64-byte rows, 64-byte
// swizzle), e.g. for bulk tensor stores from a staging tile.
inline bool make_tmap_bf16_2d_sw64(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                                   uint64_t row_stride_elems, uint32_t box_rows) {
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_stride_elems * 2};
  cuuint32_t box[2] = {32, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// A row-major byte matrix (fp8 values) [rows][cols] with a row pitch of
// `row_stride` bytes, read in boxes of box_rows x 128 bytes (128-byte swizzle).
inline bool make_tmap_u8_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                            uint64_t row_stride, uint32_t box_rows) {
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_stride};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The tiled block scales of a 4-bit matrix (h3attn_lowp.h): `groups` 128-row groups of
// `tiles` 512-byte tiles each, read in boxes of box_groups x box_tiles (at most 4) tiles,
// unswizzled; tiles past the end read as zero.  Counted in 8-byte elements: 64 a tile.
inline bool make_tmap_scales(CUtensorMap* map, const void* base, uint64_t groups, uint64_t tiles,
                             uint32_t box_groups, uint32_t box_tiles) {
  cuuint64_t dims[2] = {tiles * 64, groups};
  cuuint64_t strides[1] = {tiles * 512};
  cuuint32_t box[2] = {box_tiles * 64, box_groups};
  cuuint32_t estr[2] = {1, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 2, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace h3
