// Host-side TMA tensor-map encoding through the driver entry point obtained
// from the runtime (the library does not link libcuda directly, so it still
// loads on machines without a driver).
#include <cudaTypedefs.h>

#include <atomic>

#include "tc.cuh"

namespace csa {

namespace {

// A tiled map of a 2-D tensor: `cols` x `rows` elements, boxes of box_cols x box_rows.
bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t rows, uint64_t cols,
               uint64_t row_stride_bytes, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  static std::atomic<void*> known{nullptr};
  void* fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return false;
    known.store(fn, std::memory_order_relaxed);
  }
  const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_stride_bytes};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  auto call = [&] {
    return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = call();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // A host thread that has made no runtime call yet has no current context, and the driver call does not make one:
    // the runtime binds the device's own to the thread.
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
    r = call();
  }
  return r == CUDA_SUCCESS;
}

}  // namespace

bool make_tmap_2d_bf16(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t row_stride_bytes,
                       uint32_t box_rows) {
  if ((reinterpret_cast<uintptr_t>(base) & 15u) || (row_stride_bytes & 15u) || box_rows == 0 || box_rows > 256)
    return false;
  return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rows, cols, row_stride_bytes, 64, box_rows,
                   CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_tmap_2d_u8(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t row_stride_bytes,
                     uint32_t box_cols, uint32_t box_rows, bool swizzle128) {
  if ((reinterpret_cast<uintptr_t>(base) & 15u) || (row_stride_bytes & 15u) || box_rows == 0 || box_rows > 256 ||
      box_cols == 0 || (box_cols & 15u) || box_cols > (swizzle128 ? 128u : 256u) || cols < box_cols)
    return false;
  return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rows, cols, row_stride_bytes, box_cols, box_rows,
                   swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace csa
