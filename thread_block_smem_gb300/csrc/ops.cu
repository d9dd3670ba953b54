// ops.cu -- host-side helpers of the linear-layer operators (ops.h).
#include "ops.h"

#include <mutex>

#include "common.h"

namespace swz {

__device__ unsigned int g_op_status_word;  // nonzero: a bounded wait expired

int op_status_word(unsigned int** word) {
  static std::mutex mu;
  static unsigned int* cache[64] = {};
  int dev = 0;
  SWZ_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return SWZ_EINVAL;
  std::lock_guard<std::mutex> lock(mu);
  if (!cache[dev]) {
    void* p = nullptr;
    SWZ_CUDA_TRY(cudaGetSymbolAddress(&p, g_op_status_word));
    cache[dev] = static_cast<unsigned int*>(p);
  }
  *word = cache[dev];
  return SWZ_OK;
}

int take_op_status(bool* expired) {
  unsigned int v = 0;
  SWZ_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_op_status_word, sizeof(v)));
  *expired = v != 0;
  if (v != 0) {
    const unsigned int zero = 0;
    SWZ_CUDA_TRY(cudaMemcpyToSymbol(g_op_status_word, &zero, sizeof(zero)));
  }
  return SWZ_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

int encode_bytes(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld,
                 uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cuda_fail(cudaErrorNotSupported);
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {ld};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SWZ_OK : cuda_fail(cudaErrorInvalidValue);
}

int encode_half(CUtensorMap* map, const void* base, uint64_t batch, uint64_t rows, uint64_t cols,
                uint64_t ld, uint64_t batch_stride, uint32_t box_cols, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cuda_fail(cudaErrorNotSupported);
  const cuuint64_t dims[3] = {cols, rows, batch};
  const cuuint64_t strides[2] = {ld * 2, batch_stride * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box,
         estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SWZ_OK : cuda_fail(cudaErrorInvalidValue);
}

}  // namespace swz
