// int8.cuh -- what the parts of the 8-bit integer product share.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rows.cuh"

namespace swz {
namespace i8 {

// Longest K: 131071 products of magnitude 2^14 or less stay below 2^31.
constexpr int kMaxK = 131071;

// Rows of x to whole numbers -127 .. 127 and a scale each (arguments checked by the
// caller): as bytes, or as fp16 numbers of the same values (ldq in bytes; whole
// chunks of eight values are written).
int quantize_rows(const void* x, int dtype, int64_t ldx, int M, int K, void* q, int64_t ldq,
                  float* scales, bool half, cudaStream_t s);

// The product of up to kTokens rows of A (bytes with the scales sa), or with A NULL
// the layer of as many rows of x (tokens_fused says where); arguments checked by the
// caller.
constexpr int kTokens = 2;
bool tokens_fused(int M, int K);
int gemm_int8_tokens(const void* A, int64_t lda, const float* sa, const void* x, int x_dtype,
                     int64_t ldx, const void* B, int64_t ldb, const float* sb, void* C,
                     int64_t ldc, int c_dtype, int M, int N, int K, int num_sms,
                     cudaStream_t stream);

// The product of up to kRingRows rows of A, which needs no workspace (split 0:
// automatic).  `early_b`: the kernel before in the stream is the quantiser of A,
// launched by the same call, and B may be read while it runs.
constexpr int kRingRows = 32;
int gemm_int8_rows(const void* A, int64_t lda, const float* sa, const void* B, int64_t ldb,
                   const float* sb, void* C, int64_t ldc, int c_dtype, int M, int N, int K,
                   int split, uint32_t debug_flags, uint64_t timeout_ns, bool early_b,
                   int num_sms, cudaStream_t stream);

// The product of a few to some hundred rows of A, given as fp16 numbers (rows of `ld`
// elements, written by the kernel that the same call launched before), with B as
// bytes; arguments checked by the caller.
constexpr int kBatchRows = 512;
struct BatchPlan {
  uint32_t tiles_m, nb, ctas_per_sm, stages, slots, split, tmem_cols;  // split 0: not for it
  uint64_t tiles;
};
BatchPlan batch_plan(int M, int N, int K, int split, int num_sms);
int gemm_int8_batch(const void* a16, int64_t ld, const float* sa, const void* B, int64_t ldb,
                    const float* sb, void* C, int64_t ldc, int c_dtype, int M, int N, int K,
                    const BatchPlan& b, uint32_t debug_flags, uint64_t timeout_ns,
                    cudaStream_t stream);

// 16 bytes of a row from k < K on.  What lies between K and the next multiple of 16
// is in the row as well (it may be anything: x is zero there), but for the last row
// of the matrix, whose bytes at K and beyond read as zero.
__device__ __forceinline__ uint4 load_bytes(const uint8_t* row, int k, int K, bool last) {
  if (k + 16 <= K || !last) return *reinterpret_cast<const uint4*>(row + k);
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int e = K - k - 1; e >= 0; --e) {
    hi = (hi << 8) | (lo >> 56);
    lo = (lo << 8) | row[k + e];
  }
  return make_uint4(uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32));
}

// ---- the quantisation's rule -----------------------------------------------------
// largest magnitude of a chunk of eight values, as bits of the type
template <typename T>
__device__ __forceinline__ uint32_t chunk_max(const uint32_t* w) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < T::kWords; ++j) m = f8::max_packed<T>(m, w[j] & T::kAbs);
  if constexpr (T::kBytes == 2) m = max(m & 0xFFFFu, m >> 16);
  return m;
}

// eight values to q at p: the first n as bytes, or all as fp16 numbers of the same values
template <typename T, bool HALF>
__device__ __forceinline__ void store_q(uint8_t* p, int64_t n, const uint32_t* w, float r,
                                        bool bad) {
  constexpr float kMagic = 12582912.0f;  // 1.5 2^23
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    b[i] = bad ? __float_as_uint(kMagic) : __float_as_uint(__fmaf_rn(T::value(w, i), r, kMagic));
  if constexpr (HALF) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(__uint_as_float(b[2 * i]) - kMagic,
                                          __uint_as_float(b[2 * i + 1]) - kMagic);
      o[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      o[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                         __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
    if (n >= 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
    } else {
      uint64_t v = (uint64_t(o[1]) << 32) | o[0];
#pragma unroll 1
      for (int i = 0; i < int(n); ++i, v >>= 8) p[i] = uint8_t(v);
    }
  }
}

// r and scale of a row from the bits of its largest magnitude; true where that is an
// infinity or NaN: then the scale is NaN and the row's numbers are zeros.
__device__ __forceinline__ bool row_scale(uint32_t amax_bits, float& r, float& scale) {
  f8::scale_of(amax_bits, 127.0f, r, scale);
  const bool bad = amax_bits >= 0x7F800000u;
  if (bad) scale = __uint_as_float(0x7FC00000u);
  return bad;
}

// Four bytes to four fp16 numbers of the same values: byte + 128 in the low bits of
// 1024's fp16 pattern is 1152 + the value.
__device__ __forceinline__ void widen4(uint32_t b, uint32_t& lo, uint32_t& hi) {
  b ^= 0x80808080u;
  const uint32_t bias = 0x64806480u;  // 1152 twice
  const uint32_t l = __byte_perm(b, 0x64646464u, 0x4140), h = __byte_perm(b, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&l),
                            *reinterpret_cast<const __half2*>(&bias));
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&h),
                            *reinterpret_cast<const __half2*>(&bias));
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

}  // namespace i8
}  // namespace swz
