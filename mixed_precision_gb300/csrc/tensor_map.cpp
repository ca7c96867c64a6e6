// Tensor maps for the tiled TMA loads of the block operators' kernels.
#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace zg {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, found through the runtime (the library does not link
// the driver). Looked up once; racing threads store the same address.
static EncodeFn encoder() {
  static std::atomic<void*> found{nullptr};
  void* f = found.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    found.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(f);
}

bool make_tensor_map(CUtensorMap* map, const void* base, int dtype, int dims, const uint64_t* extent,
                     const uint64_t* strides, uint32_t box_rows) {
  EncodeFn encode = encoder();
  if (encode == nullptr) return false;
  const CUtensorMapDataType type = dtype == kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint32_t box[4] = {dtype == kF32 ? 32u : 64u, box_rows, 1, 1}, step[4] = {1, 1, 1, 1};
  cuuint64_t n[4], s[3];
  for (int i = 0; i < dims; ++i) n[i] = extent[i];
  for (int i = 0; i + 1 < dims; ++i) s[i] = strides[i];
  return encode(map, type, dims, const_cast<void*>(base), n, s, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace zg
