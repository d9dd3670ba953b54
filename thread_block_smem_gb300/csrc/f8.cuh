// f8.cuh -- the 8-bit block quantisation rule, and the loads of eight values
// that the quantiser and the orthogonalisation share.
//
// A block of 128 (or 128 x 128) values with largest magnitude `amax` is held
// as q = rn_f8(x * r) with
//     ac = max(amax, 2^-96),  r = F / ac,  scale = ac / F
// both rounded to fp32; F = 448 (e4m3) or 57344 (e5m2).  x * r is at most
// F (1 + 2^-23), which rounds to F.  The bound 2^-96 keeps r finite and scale
// normal; a block of zeros gets q = 0.  amax is taken on the bit patterns of
// |x|, which order as the values do with infinity and NaN above them: a block
// with an infinity gets scale infinity and q = 0 (NaN at the infinities), one
// with a NaN gets NaN throughout, so either reads back as not finite.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "swz.h"

namespace swz {
namespace f8 {

constexpr int kBlock = 128;
constexpr uint32_t kAcMinBits = 0x0F800000u;  // 2^-96

__host__ __device__ constexpr float top(int fmt) { return fmt == SWZ_E4M3 ? 448.0f : 57344.0f; }

// scale and reciprocal of a block from the bits of its largest magnitude
__device__ __forceinline__ void scale_of(uint32_t amax_bits, float F, float& r, float& scale) {
  const float ac = __uint_as_float(amax_bits > kAcMinBits ? amax_bits : kAcMinBits);
  r = __fdiv_rn(F, ac);
  scale = __fdiv_rn(ac, F);
}

// four values to four bytes, the first in the lowest
template <int FMT>
__device__ __forceinline__ uint32_t to_f8x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  if constexpr (FMT == SWZ_E4M3) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  } else {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  }
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

// ---- input types ----------------------------------------------------------------
// kWords 32-bit words hold eight values; value(w, i) is the i-th as fp32.
// Magnitudes are compared as bit patterns, two at a time for the 16-bit types.
struct Bf16 {
  static constexpr int kBytes = 2, kWords = 4;
  static constexpr uint32_t kAbs = 0x7FFF7FFFu;
  static __device__ __forceinline__ float value(const uint32_t* w, int i) {
    return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t h) { return h << 16; }
};
struct F16 {
  static constexpr int kBytes = 2, kWords = 4;
  static constexpr uint32_t kAbs = 0x7FFF7FFFu;
  static __device__ __forceinline__ float value(const uint32_t* w, int i) {
    return __half2float(__ushort_as_half(uint16_t((i & 1) ? w[i / 2] >> 16 : w[i / 2])));
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t h) {
    return __float_as_uint(__half2float(__ushort_as_half(uint16_t(h))));
  }
};
struct F32 {
  static constexpr int kBytes = 4, kWords = 8;
  static constexpr uint32_t kAbs = 0x7FFFFFFFu;
  static __device__ __forceinline__ float value(const uint32_t* w, int i) {
    return __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t b) { return b; }
};

// the larger magnitude(s) of packed words already stripped of their signs
template <typename T>
__device__ __forceinline__ uint32_t max_packed(uint32_t a, uint32_t b) {
  if constexpr (T::kBytes == 2) return __vmaxu2(a, b);
  return a > b ? a : b;
}

// Loads eight values of a row starting at p: `n` of them exist (<= 0: none),
// the rest read as zero.  `wide`: p is 16-byte aligned when n >= 8.  Plain
// loads: the kernel before, which may still run when this one starts, may write
// what they read, and loads through the read-only path need not stay behind the
// wait for it.
template <typename T>
__device__ __forceinline__ void load8(const uint8_t* p, int n, bool wide, uint32_t* w) {
  if (n >= 8 && wide) {
#pragma unroll
    for (int j = 0; j < T::kWords / 4; ++j) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[j];
      w[4 * j] = v.x;
      w[4 * j + 1] = v.y;
      w[4 * j + 2] = v.z;
      w[4 * j + 3] = v.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < T::kWords; ++j) w[j] = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) {
      if constexpr (T::kBytes == 2)
        w[i / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i & 1));
      else
        w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    }
}

}  // namespace f8
}  // namespace swz
