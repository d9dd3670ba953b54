// layer_norm.cuh -- pieces of the layer norm's kernels.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.h"
#include "rows.cuh"

namespace swz {
namespace norm {

// A vector along a row (weight or bias): NULL reads as `none`.
struct Vec {
  const uint8_t* p;
  int dtype;
  int wide;  // 16-byte aligned
};

// Its values k .. k + 7 as fp32; those at n and beyond read as zero.
__device__ __forceinline__ void load_vec(const Vec& v, int64_t k, int64_t n, float none,
                                         float (&o)[8]) {
  if (!v.p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = none;
    return;
  }
  if (v.wide && k + 8 <= n) {
    uint32_t w[8];
    if (v.dtype == SWZ_F32) {
      rows::ld16(v.p + k * 4, w);
      rows::ld16(v.p + k * 4 + 16, w + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rows::F32::value(w, i);
    } else {
      rows::ld16(v.p + k * 2, w);
      if (v.dtype == SWZ_BF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rows::Bf16::value(w, i);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rows::F16::value(w, i);
      }
    }
    return;
  }
  const int es = v.dtype == SWZ_F32 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = k + i < n ? rows::load1(v.p + (k + i) * es, v.dtype) : 0.0f;
}

inline bool float_type(int d) { return d == SWZ_F16 || d == SWZ_BF16 || d == SWZ_F32; }
inline int64_t size_of(int d) { return d == SWZ_F32 ? 4 : 2; }

inline Vec vec(const void* p, int dtype) {
  Vec v{};
  v.p = static_cast<const uint8_t*>(p);
  v.dtype = dtype;
  v.wide = aligned16(p);
  return v;
}

// M rows of N values at p, or none of them wanted
inline bool matrix_ok(const void* p, int dtype, int64_t ld, int M, int N) {
  return p && reinterpret_cast<uintptr_t>(p) % uintptr_t(size_of(dtype)) == 0 &&
         (M <= 1 || ld >= N);
}
inline bool vector_ok(const void* p, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % uintptr_t(size_of(dtype)) == 0;
}

template <typename Kernel, typename Args>
int launch(Kernel k, uint32_t grid, uint32_t threads, const Args& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, k, a));
  return SWZ_OK;
}

}  // namespace norm
}  // namespace swz
