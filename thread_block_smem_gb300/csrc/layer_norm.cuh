// layer_norm.cuh -- pieces of the layer norm's kernels.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "common.h"
#include "pipe.cuh"
#include "rows.cuh"

namespace swz {
namespace norm {

// A vector along a row (weight or bias): NULL reads as `none`.
struct Vec {
  const uint8_t* p;
  int dtype;
  int wide;  // 16-byte aligned
};

// Its values k .. k + 7 one by one.
__device__ __forceinline__ rows::Eight load_vec_some(Vec v, int64_t k, int64_t n) {
  const int es = v.dtype == SWZ_F32 ? 4 : 2;
  rows::Eight e;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    e.v[i] = k + i < n ? rows::load1(v.p + (k + i) * es, v.dtype) : 0.0f;
  return e;
}

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
  const rows::Eight e = load_vec_some(v, k, n);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = e.v[i];
}

// ---- chunks as pairs of fp32 values ---------------------------------------------------
// Arithmetic is packed, two values an instruction: with one at a time the kernels were
// bound by their instructions, not by memory.
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float v) { return pipe::pack2(v, v); }
__device__ __forceinline__ float sum_of(uint64_t v) {
  float a, b;
  pipe::unpack2(v, a, b);
  return a + b;
}

template <typename T>
__device__ __forceinline__ void pairs_of(const uint32_t* w, uint64_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pipe::pack2(T::value(w, 2 * i), T::value(w, 2 * i + 1));
}

__device__ __forceinline__ void load_vec2(const Vec& v, int64_t k, int64_t n, float none,
                                          uint64_t (&o)[4]) {
  float f[8];
  load_vec(v, k, n, none, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pipe::pack2(f[2 * i], f[2 * i + 1]);
}

__device__ __forceinline__ void store_pairs(uint8_t* p, int64_t n, const uint64_t (&o)[4], int dtype,
                                            bool wide) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) pipe::unpack2(o[i], f[2 * i], f[2 * i + 1]);
  rows::store8(p, n, f, dtype, wide);
}

// ---- the common case ------------------------------------------------------------------
// Rows that start on 16 bytes and have whole chunks, weight and bias of one kind (G = 1
// fp32, G = 2 the type of x, 16-bit), results of the type of x: nothing to ask per chunk.
// The general form (G = 0), whose chunks may be cut, shifted and of any type, executes
// three times the instructions.
template <typename T>
__device__ __forceinline__ void fast_load(const uint8_t* p, bool in, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < T::kWords; ++j) w[j] = 0u;
  if (in)
#pragma unroll
    for (int j = 0; j < T::kWords / 4; ++j) rows::ld16_once(p + 16 * j, w + 4 * j);
}

template <typename T, int G>
__device__ __forceinline__ void fast_vec(const uint8_t* p, int k, uint64_t (&o)[4]) {
  if constexpr (G == 1) {
    const ulonglong2* q = reinterpret_cast<const ulonglong2*>(p + int64_t(k) * 4);
    const ulonglong2 a = q[0], b = q[1];
    o[0] = a.x;
    o[1] = a.y;
    o[2] = b.x;
    o[3] = b.y;
  } else {
    uint32_t w[8];
    rows::ld16(p + int64_t(k) * 2, w);
    pairs_of<T>(w, o);
  }
}

template <typename T>
__device__ __forceinline__ void fast_store(uint8_t* p, const uint64_t (&o)[4]) {
  if constexpr (T::kBytes == 4) {
    reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(o[0], o[1]);
    reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(o[2], o[3]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      pipe::unpack2(o[i], a, b);
      w[i] = rows::pack16(a, b, std::is_same<T, rows::Bf16>::value ? SWZ_BF16 : SWZ_F16);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

inline bool float_type(int d) { return d == SWZ_F16 || d == SWZ_BF16 || d == SWZ_F32; }
inline int64_t size_of(int d) { return d == SWZ_F32 ? 4 : 2; }

template <typename T>
constexpr int code_of() {
  return T::kBytes == 4 ? int(SWZ_F32)
                        : std::is_same<T, rows::Bf16>::value ? int(SWZ_BF16) : int(SWZ_F16);
}

// G of a weight (and bias) beside rows of type T
template <typename T>
int kind_of(const Vec& a) {
  if (!a.p || !a.wide) return 0;
  return a.dtype == SWZ_F32 ? 1 : a.dtype == code_of<T>() ? 2 : 0;
}

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

// Whether a result may be written while an input is read: nothing in common, or the same
// rows of the same type, which are read before they are written.
inline RowsInMemory rows_at(const void* p, int dtype, int64_t ld, int M, int N) {
  const int64_t es = size_of(dtype);
  return RowsInMemory{p, M, (M > 1 ? ld : int64_t(N)) * es, int64_t(N) * es};
}
inline bool may_lie(const RowsInMemory& result, int result_dtype, const RowsInMemory& input,
                    int input_dtype) {
  return (result.p == input.p && result_dtype == input_dtype && result.ld == input.ld) ||
         !rows_meet(result, input);
}
inline bool apart(const RowsInMemory& result, const void* values, int64_t bytes) {
  return !values || !rows_meet(result, RowsInMemory{values, 1, bytes, bytes});
}

// Threads of a CTA whose threads hold nc chunks of a row of N values each.
inline int threads_of(int N, int nc) {
  return int((int64_t(N) + int64_t(nc) * 256 - 1) / (int64_t(nc) * 256)) * 32;
}

// CTAs of `threads` threads (512 at most) that stay on an SM, looked up once.
template <auto K>
int resident_ctas(int threads, int* n) {
  static std::atomic<int> cache[17];  // this kernel's, by warps
  std::atomic<int>& at = cache[threads / 32];
  *n = at.load(std::memory_order_relaxed);
  if (*n == 0) {
    SWZ_CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, K, threads, 0));
    if (*n < 1) *n = 1;
    at.store(*n, std::memory_order_relaxed);
  }
  return SWZ_OK;
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
