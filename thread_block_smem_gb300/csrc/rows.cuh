// rows.cuh -- what the kernels that work along rows share (8-bit quantisation by
// rows, layer norm, gradient norm): eight values at a time to and from rows that
// start anywhere, and sums and maxima over a row's threads.
//
// A thread owns "chunks" of eight consecutive values, consecutive lanes
// consecutive chunks.  Where rows start on 16 bytes a chunk is one or two 16-byte
// accesses.  Where they do not (an odd width in 16 bits, a view), value by value
// a warp's access would touch eight times the sectors; so a load takes the
// aligned 16-byte pieces around the chunk and shifts, and a store exchanges with
// the lane before and writes aligned pieces, all but the ends of the warp's part.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "f8.cuh"

namespace swz {
namespace rows {

using f8::Bf16;
using f8::F16;
using f8::F32;

// A matrix as the kernels read it: base, bytes from row to row, and the end of
// its last row (no load touches a byte outside base .. end).
struct Span {
  const uint8_t* base;
  const uint8_t* end;
  int64_t ld;  // bytes
  int wide;    // every row starts on 16 bytes
};

// M rows of N values of a type (SWZ_F16, ...), `ld` elements apart.
inline Span span_of(const void* x, int dtype, int64_t ld, int M, int N) {
  const int64_t es = dtype == SWZ_F32 ? 4 : 2;
  Span s{};
  s.base = static_cast<const uint8_t*>(x);
  s.ld = (M > 1 ? ld : int64_t(N)) * es;
  s.end = s.base + (int64_t(M) - 1) * s.ld + int64_t(N) * es;
  s.wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 && s.ld % 16 == 0;
  return s;
}

// The 16-byte piece at byte `s` (1 .. 15, the same for all its words) of the words
// e[0..7].
__device__ __forceinline__ void shift_words(const uint32_t (&e)[8], uint32_t s, uint32_t* o) {
  uint32_t a[6], b[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) a[i] = (s & 8u) ? e[i + 2] : e[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) b[i] = (s & 4u) ? a[i + 1] : a[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (s & 2u) ? __funnelshift_r(b[i], b[i + 1], 16) : b[i];
}

__device__ __forceinline__ void ld16(const uint8_t* p, uint32_t* w) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  w[0] = v.x;
  w[1] = v.y;
  w[2] = v.z;
  w[3] = v.w;
}

// The same, of what is read once: it leaves L1 to what is read again.
__device__ __forceinline__ void ld16_once(const uint8_t* p, uint32_t* w) {
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p)
               : "memory");
}

// Four words of the first n values at p, from the value `from` on (16-bit: all eight).
// In loops, as the other rare paths are: unrolled into each chunk they made kernels of
// a few rows wait for their instructions.
template <typename T>
__device__ __forceinline__ uint4 load_some(const uint8_t* p, int n, int from) {
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int i = 7; i >= 0; --i) {
    const bool in = i < n;
    if constexpr (T::kBytes == 2) {
      hi = (hi << 16) | (lo >> 48);
      lo = (lo << 16) | (in ? uint64_t(reinterpret_cast<const uint16_t*>(p)[i]) : 0u);
    } else if (i >= from && i < from + 4) {
      hi = (hi << 32) | (lo >> 32);
      lo = (lo << 32) | (in ? uint64_t(reinterpret_cast<const uint32_t*>(p)[i]) : 0u);
    }
  }
  return make_uint4(uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32));
}

// Eight values at p, of which `n` exist (<= 0: none); the others read as zero.
// Plain loads: what they read may be written by the kernel before, which may
// still run when this one starts.
template <typename T, bool ONCE = false>
__device__ __forceinline__ void load8(const uint8_t* p, int64_t n, const Span& m, uint32_t* w) {
  if (n >= 8) {
    const uint32_t s = m.wide ? 0u : uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u;
    if (s == 0) {
#pragma unroll
      for (int j = 0; j < T::kWords / 4; ++j) {
        if constexpr (ONCE) ld16_once(p + 16 * j, w + 4 * j);
        else ld16(p + 16 * j, w + 4 * j);
      }
      return;
    }
    const uint8_t* q = p - s;
    if (q >= m.base && q + T::kBytes * 8 + 16 <= m.end) {
      uint32_t e[T::kWords + 4];
#pragma unroll
      for (int j = 0; j < T::kWords / 4 + 1; ++j) ld16(q + 16 * j, e + 4 * j);
#pragma unroll
      for (int j = 0; j < T::kWords / 4; ++j) {
        const uint32_t f[8] = {e[4 * j],     e[4 * j + 1], e[4 * j + 2], e[4 * j + 3],
                               e[4 * j + 4], e[4 * j + 5], e[4 * j + 6], e[4 * j + 7]};
        shift_words(f, s, w + 4 * j);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < T::kWords; ++j) w[j] = 0u;
  if (n > 0) {
    const int some = n < 8 ? int(n) : 8;
#pragma unroll
    for (int j = 0; j < T::kWords / 4; ++j) {
      const uint4 v = load_some<T>(p, some, 4 * j);
      w[4 * j] = v.x;
      w[4 * j + 1] = v.y;
      w[4 * j + 2] = v.z;
      w[4 * j + 3] = v.w;
    }
  }
}

template <typename T>
__device__ __forceinline__ void load8_once(const uint8_t* p, int64_t n, const Span& m,
                                           uint32_t* w) {
  load8<T, true>(p, n, m, w);
}

__device__ __forceinline__ uint32_t pack16(float a, float b, int dtype) {
  if (dtype == SWZ_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store1(uint8_t* p, float v, int dtype) {
  if (dtype == SWZ_F32) *reinterpret_cast<float*>(p) = v;
  else if (dtype == SWZ_BF16) *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v);
  else *reinterpret_cast<__half*>(p) = __float2half_rn(v);
}

__device__ __forceinline__ float load1(const uint8_t* p, int dtype) {
  if (dtype == SWZ_F32) return *reinterpret_cast<const float*>(p);
  if (dtype == SWZ_BF16) return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
  return __half2float(*reinterpret_cast<const __half*>(p));
}

// The values from .. to - 1 of v at p, one by one.
struct Eight {
  float v[8];
};
__device__ __forceinline__ void store_some(uint8_t* p, Eight e, int from, int to, int dtype) {
  const int es = dtype == SWZ_F32 ? 4 : 2;
#pragma unroll 1
  for (int i = from; i < to; ++i) {
    float x = e.v[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) x = i == j ? e.v[j] : x;
    store1(p + i * es, x, dtype);
  }
}

// Stores `n` (unclamped: 8 or more for a whole chunk, <= 0 for none) of the eight
// values v at p, rounded once.  All lanes of the warp call it together, lane i with
// the chunk after lane i - 1's.
__device__ __forceinline__ void store8(uint8_t* p, int64_t n, const float (&v)[8], int dtype,
                                       bool wide) {
  const uint32_t lane = threadIdx.x & 31u;
  const bool f32 = dtype == SWZ_F32;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
  if (!f32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack16(v[2 * i], v[2 * i + 1], dtype);
  }
  const uint32_t s = wide ? 0u : uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u;  // uniform
  if (s == 0) {
    if (n >= 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      if (f32) *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
      return;
    }
    if (n > 0) {
      Eight x;
#pragma unroll
      for (int i = 0; i < 8; ++i) x.v[i] = v[i];
      store_some(p, x, 0, int(n), dtype);
    }
    return;
  }
  // the last 16 bytes of the lane before, then this lane's: `head` bytes of its own
  // complete the piece that the lane before began
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = __shfl_up_sync(0xFFFFFFFFu, f32 ? w[4 + i] : w[i], 1);
    e[4 + i] = w[i];
  }
  const int es = f32 ? 4 : 2, head = int(16u - s) / es, last = int(s) / es;
  // first: the piece at p - s; for fp32 a second one that is this lane's alone
  const bool full = lane > 0 && n >= head;
  const int whole = 8 - last;  // values before the last, begun piece
  uint32_t o[4];
  shift_words(e, 16u - s, o);
  if (full) *reinterpret_cast<uint4*>(p - s) = make_uint4(o[0], o[1], o[2], o[3]);
  int from = full ? head : 0;  // values from here on are not stored yet
  if (f32 && full && n >= whole) {
    const uint32_t g[8] = {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
    shift_words(g, 16u - s, o);
    *reinterpret_cast<uint4*>(p + (16u - s)) = make_uint4(o[0], o[1], o[2], o[3]);
    from = whole;
  }
  // the next lane stores this one's last values with its own head, if it is full
  const int to = (lane < 31 && n - 8 >= head) ? whole : 8;
  const int end = n < to ? int(n) : to;
  if (from < end) {
    Eight x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.v[i] = v[i];
    store_some(p, x, from, end, dtype);
  }
}

// Sum of v over the warp, the same bits in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// Sums over the TPR threads of a row (a warp, or the whole CTA).  `part`: TPR / 32
// values of shared memory for each of the K sums, free to be overwritten; the same
// bits in every thread.
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* part) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) part[k * W + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = part[k * W];
#pragma unroll
      for (int i = 1; i < W; ++i) v[k] += part[k * W + i];
    }
  }
}

}  // namespace rows
}  // namespace swz
