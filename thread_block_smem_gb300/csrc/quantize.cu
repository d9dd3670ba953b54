// quantize.cu -- block quantisation to 8 bits (rule in f8.cuh): x (M x K) by
// blocks of 1 x 128 along its rows or of 128 x 128, and the same of x^T (the
// operand of a gradient's product), in one read of x.
//
// Bound: memory.  One CTA takes a 128 x 128 block of x: thread (g, c) = (t /
// 16, t % 16) holds rows 8g .. 8g+7, columns 8c .. 8c+7 as loaded.  A row of
// the block is 16 lanes of one half-warp, so its maximum takes four shuffles
// (two 16-bit rows at a time); a thread's eight rows of one column are eight
// consecutive bytes of x^T's row, so the transpose goes through shared memory
// as 8-byte words (16 KB, 16-byte chunk index XORed with the column group so
// that neither side has bank conflicts) and leaves as 16-byte stores.
//
// Measured (bytes read and written; the copy bandwidth is 6.8 TB/s): 8192 x 4096
// bf16 with x^T, square blocks 22.6 us (5.9 TB/s), row blocks 26.1 (5.1);
// 8192 x 8192 42.1 (6.4) and 45.9 (5.8), row blocks without x^T 34.6 to 37.2 (5.5 to
// 5.9); 10240 x 4096 fp32, square, 38.3 (6.6).
// Row blocks keep a scale for each of a thread's 8 rows and 8 columns and
// exchange maxima along both: 64 registers against 48, 44 % of the warps
// resident, and the loads of the next blocks wait for the arithmetic of these.
#include "common.h"
#include "f8.cuh"
#include "ptx.cuh"

namespace swz {
namespace f8 {

struct QuantArgs {
  const uint8_t* x;
  int64_t ldx;  // elements
  int M, K;
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t lds;
  uint8_t* qt;
  int64_t ldqt;
  float* st;
  int64_t ldst;
  int wide;  // rows of x start on 16 bytes
  uint32_t col_blocks;
};

template <typename T, bool SQUARE, int FMT>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs p) {
  __shared__ uint4 tile[128 * 8];       // x^T in 8 bits: 128 columns x 128 bytes
  __shared__ uint32_t part[8][128];     // column maxima by warp (packed for 16-bit types)
  __shared__ float rcol[128];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t t = threadIdx.x, c = t & 15u, g = t >> 4, warp = t >> 5, lane = t & 31u;
  const uint32_t kb = blockIdx.x % p.col_blocks, mb = blockIdx.x / p.col_blocks;
  const int k0 = int(kb) * kBlock + int(c) * 8, m0 = int(mb) * kBlock + int(g) * 8;
  constexpr float F = top(FMT);

  uint32_t w[8][T::kWords];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load8<T>(p.x + (int64_t(m0 + i) * p.ldx + k0) * T::kBytes, m0 + i < p.M ? p.K - k0 : 0,
             p.wide != 0, w[i]);

  // maxima of this thread's rows and columns, as bits
  uint32_t rmax[8];                 // row i of the thread
  uint32_t cmax[T::kWords];         // its columns, packed as the words are
#pragma unroll
  for (int j = 0; j < T::kWords; ++j) cmax[j] = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < T::kWords; ++j) {
      const uint32_t a = w[i][j] & T::kAbs;
      m = max_packed<T>(m, a);
      cmax[j] = max_packed<T>(cmax[j], a);
    }
    if constexpr (T::kBytes == 2) m = max(m & 0xFFFFu, m >> 16);
    rmax[i] = m;
  }

  float rr[8];  // 1 / scale of each row (of the block when SQUARE)
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rmax[i]);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) part[warp][0] = m;
    __syncthreads();
    m = part[0][0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = max(m, part[j][0]);
    float r, scale;
    scale_of(T::max_bits(m), F, r, scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) rr[i] = r;
    if (t == 0) {
      if (p.q) p.s[int64_t(mb) * p.lds + kb] = scale;
      if (p.qt) p.st[int64_t(kb) * p.ldst + mb] = scale;
    }
  } else if (p.q) {
    if constexpr (T::kBytes == 2) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        uint32_t two = rmax[i] | (rmax[i + 1] << 16);
#pragma unroll
        for (int d = 1; d < 16; d *= 2) two = __vmaxu2(two, __shfl_xor_sync(0xFFFFFFFFu, two, d));
        rmax[i] = two & 0xFFFFu;
        rmax[i + 1] = two >> 16;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int d = 1; d < 16; d *= 2)
          rmax[i] = max(rmax[i], __shfl_xor_sync(0xFFFFFFFFu, rmax[i], d));
    }
    // lane c of a row group works out row c's scale (c < 8), the others read it
    uint32_t mine = rmax[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mine = (c & 7u) == uint32_t(i) ? rmax[i] : mine;
    float r, scale;
    scale_of(T::max_bits(mine), F, r, scale);
    if (c < 8u && m0 + int(c) < p.M) p.s[int64_t(kb) * p.lds + m0 + int(c)] = scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) rr[i] = __shfl_sync(0xFFFFFFFFu, r, i, 16);
  }

  if (p.q && k0 < p.K) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (m0 + i >= p.M) break;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = T::value(w[i], j) * rr[i];
      uint2 o;
      o.x = to_f8x4<FMT>(v[0], v[1], v[2], v[3]);
      o.y = to_f8x4<FMT>(v[4], v[5], v[6], v[7]);
      *reinterpret_cast<uint2*>(p.q + int64_t(m0 + i) * p.ldq + k0) = o;
    }
  }
  if (!p.qt) return;

  float rc[8];  // 1 / scale of each column
  if constexpr (!SQUARE) {
    // columns: the two row groups of the warp, then the eight warps
#pragma unroll
    for (int j = 0; j < T::kWords; ++j) {
      cmax[j] = max_packed<T>(cmax[j], __shfl_xor_sync(0xFFFFFFFFu, cmax[j], 16));
      if (lane < 16u) part[warp][c * T::kWords + j] = cmax[j];
    }
    __syncthreads();
    if (t < 128u) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (T::kBytes == 2) {
          const uint32_t two = part[j][t / 2];
          m = max(m, (t & 1u) ? two >> 16 : two & 0xFFFFu);
        } else {
          m = max(m, part[j][t]);
        }
      }
      float r, scale;
      scale_of(T::max_bits(m), F, r, scale);
      rcol[t] = r;
      const int k = int(kb) * kBlock + int(t);
      if (k < p.K) p.st[int64_t(mb) * p.ldst + k] = scale;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) rc[j] = rcol[c * 8 + j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) rc[j] = rr[0];
  }
  // column 8c + j: this thread's rows are bytes 8g .. 8g+7 of its line
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = T::value(w[i], j) * rc[j];
    uint2 o;
    o.x = to_f8x4<FMT>(v[0], v[1], v[2], v[3]);
    o.y = to_f8x4<FMT>(v[4], v[5], v[6], v[7]);
    uint8_t* line = reinterpret_cast<uint8_t*>(tile) + (c * 8 + j) * 128;
    *reinterpret_cast<uint2*>(line + (((g >> 1) ^ (c & 7u)) << 4) + ((g & 1u) << 3)) = o;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t col = t / 8 + 32 * i, chunk = t & 7u;
    const int k = int(kb) * kBlock + int(col), m = int(mb) * kBlock + int(chunk) * 16;
    if (k < p.K && m < p.M)
      *reinterpret_cast<uint4*>(p.qt + int64_t(k) * p.ldqt + m) =
          tile[col * 8 + (chunk ^ ((col >> 3) & 7u))];
  }
}

}  // namespace f8
}  // namespace swz

using namespace swz;

template <typename T, bool SQUARE, int FMT>
static int launch_quantize(const f8::QuantArgs& a, uint32_t grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, f8::quantize_kernel<T, SQUARE, FMT>, a));
  return SWZ_OK;
}

template <typename T>
static int dispatch_quantize(const f8::QuantArgs& a, int block, int fmt, uint32_t grid,
                             cudaStream_t s) {
  if (block == SWZ_BLOCK_SQUARE)
    return fmt == SWZ_E4M3 ? launch_quantize<T, true, SWZ_E4M3>(a, grid, s)
                           : launch_quantize<T, true, SWZ_E5M2>(a, grid, s);
  return fmt == SWZ_E4M3 ? launch_quantize<T, false, SWZ_E4M3>(a, grid, s)
                         : launch_quantize<T, false, SWZ_E5M2>(a, grid, s);
}

extern "C" int swz_quantize_fp8(const void* x, int dtype, int64_t ldx, int M, int K, int block,
                                int fmt, void* q, int64_t ldq, float* scales, int64_t ld_scales,
                                void* qt, int64_t ldqt, float* scales_t, int64_t ld_scales_t,
                                void* stream) {
  if (M < 0 || K < 0) return SWZ_EINVAL;
  if (dtype != SWZ_F16 && dtype != SWZ_BF16 && dtype != SWZ_F32) return SWZ_EINVAL;
  if (block != SWZ_BLOCK_ROW && block != SWZ_BLOCK_SQUARE) return SWZ_EINVAL;
  if (fmt != SWZ_E4M3 && fmt != SWZ_E5M2) return SWZ_EINVAL;
  if (M == 0 || K == 0) return SWZ_OK;
  const int64_t kb = (int64_t(K) + f8::kBlock - 1) / f8::kBlock;
  const int64_t mb = (int64_t(M) + f8::kBlock - 1) / f8::kBlock;
  const bool square = block == SWZ_BLOCK_SQUARE;
  const int64_t es = dtype == SWZ_F32 ? 4 : 2;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x);
  if (!x || xa % uintptr_t(es) != 0 || (M > 1 && ldx < K) || ldx < 0) return SWZ_EINVAL;
  if (!q && !qt) return SWZ_EINVAL;
  if (q && (!aligned16(q) || ldq < K || ldq % 16 != 0 || !scales || !aligned4(scales) ||
            ld_scales < (square ? kb : int64_t(M))))
    return SWZ_EINVAL;
  if (qt && (!aligned16(qt) || ldqt < M || ldqt % 16 != 0 || !scales_t || !aligned4(scales_t) ||
             ld_scales_t < (square ? mb : int64_t(K))))
    return SWZ_EINVAL;
  if (kb * mb > INT32_MAX) return SWZ_EINVAL;
  DeviceInfo dev{};
  const int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  f8::QuantArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.ldx = M > 1 ? ldx : K;
  a.M = M;
  a.K = K;
  a.q = static_cast<uint8_t*>(q);
  a.ldq = ldq;
  a.s = scales;
  a.lds = ld_scales;
  a.qt = static_cast<uint8_t*>(qt);
  a.ldqt = ldqt;
  a.st = scales_t;
  a.ldst = ld_scales_t;
  a.wide = xa % 16 == 0 && (M == 1 || (a.ldx * es) % 16 == 0);
  a.col_blocks = uint32_t(kb);
  const uint32_t grid = uint32_t(kb * mb);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SWZ_BF16) return dispatch_quantize<f8::Bf16>(a, block, fmt, grid, s);
  if (dtype == SWZ_F16) return dispatch_quantize<f8::F16>(a, block, fmt, grid, s);
  return dispatch_quantize<f8::F32>(a, block, fmt, grid, s);
}
