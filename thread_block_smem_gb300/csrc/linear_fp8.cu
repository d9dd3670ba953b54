// linear_fp8.cu -- y = x W^T with W kept in 8 bits: x (M x K; fp16, bf16 or
// fp32) is quantised in row blocks (e4m3) and multiplied as swz_gemm_fp8 does.
//
// Few rows (decoding): bound by reading W once, N * K bytes.  One kernel that
// streams W and quantises x on the way: a CTA takes 16 rows of W, its 8 warps
// share the blocks of K and add their sums through shared memory at the end.
// mma.sync m16n8k32 with W as the 16-row operand: lane (g, t) = (lane / 4,
// lane mod 4) reads 16 bytes of W's rows g and g + 8 at k = 16 t (and 64 +
// 16 t) of a block -- the order of k inside a block is free as long as both
// operands share it -- and the same 32 values of row g of x, whose block
// maximum is then two shuffles away and whose 8-bit values land in the
// registers where the instruction takes them.  tcgen05 has no use here: its
// 128-row tile would be at most an eighth full and its operands would take a
// detour through shared memory.
// More rows: the quantiser into the caller's workspace, then the GEMM.
#include "common.h"
#include "f8.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace swz {
namespace f8 {

struct RowsArgs {
  const uint8_t* x;
  int64_t ldx;  // elements
  int wide;
  const uint8_t* w;
  int64_t ldw;
  const float* sw;
  int64_t ldsw;
  int w_square, w_fmt;
  void* y;
  int64_t ldy;
  int y_dtype;
  int M, N, K;
  int num_kb;
};

__device__ __forceinline__ void mma_16832(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1, int a_fmt) {
  if (a_fmt == SWZ_E4M3)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes of a row of which `n` exist: the rest are zero and not read
__device__ __forceinline__ uint4 load_bytes(const uint8_t* p, int n) {
  if (n >= 16) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < n) u[j / 4] |= uint32_t(__ldg(p + j)) << (8 * (j % 4));
  return make_uint4(u[0], u[1], u[2], u[3]);
}

constexpr int kRowsWarps = 8, kRowsUnroll = 4, kWRows = 16;

template <typename T, int MT>
__global__ void __launch_bounds__(kRowsWarps * 32) linear_rows_kernel(const RowsArgs p) {
  __shared__ float red[kRowsWarps][MT][8][kWRows];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3u;
  const int n0 = int(blockIdx.x) * kWRows;
  const int64_t r0 = int64_t(n0) + g, r1 = r0 + 8;
  const bool in0 = r0 < p.N, in1 = r1 < p.N;
  float acc[MT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[mt][j] = 0.f;

  for (int base = int(warp); base < p.num_kb; base += kRowsWarps * kRowsUnroll) {
    uint4 wv[kRowsUnroll][2][2];
    float ws[kRowsUnroll][2];
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
      const int kb = base + u * kRowsWarps;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = min(kb, p.num_kb - 1) * kBlock + h * 64 + int(t) * 16;
        const int left = kb < p.num_kb ? p.K - k : 0;
        wv[u][0][h] = load_bytes(p.w + r0 * p.ldw + k, in0 ? left : 0);
        wv[u][1][h] = load_bytes(p.w + r1 * p.ldw + k, in1 ? left : 0);
      }
      ws[u][0] = ws[u][1] = 0.f;
      if (kb < p.num_kb) {
        if (p.w_square) {
          ws[u][0] = ws[u][1] = __ldg(p.sw + int64_t(n0 / kBlock) * p.ldsw + kb);
        } else {
          if (in0) ws[u][0] = __ldg(p.sw + int64_t(kb) * p.ldsw + r0);
          if (in1) ws[u][1] = __ldg(p.sw + int64_t(kb) * p.ldsw + r1);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
      const int kb = base + u * kRowsWarps;
      if (kb >= p.num_kb) break;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int row = mt * 8 + int(g);
        uint32_t xw[4][T::kWords];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = kb * kBlock + (j >> 1) * 64 + int(t) * 16 + (j & 1) * 8;
          load8<T>(p.x + (int64_t(row) * p.ldx + k) * T::kBytes, row < p.M ? p.K - k : 0,
                   p.wide != 0, xw[j]);
#pragma unroll
          for (int i = 0; i < T::kWords; ++i) m = max_packed<T>(m, xw[j][i] & T::kAbs);
        }
        if constexpr (T::kBytes == 2) m = max(m & 0xFFFFu, m >> 16);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        float r, scale;
        scale_of(T::max_bits(m), top(SWZ_E4M3), r, scale);
        uint32_t x8[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            x8[j >> 1][(j & 1) * 2 + i] =
                to_f8x4<SWZ_E4M3>(T::value(xw[j], 4 * i) * r, T::value(xw[j], 4 * i + 1) * r,
                                  T::value(xw[j], 4 * i + 2) * r, T::value(xw[j], 4 * i + 3) * r);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 a = wv[u][0][h], b = wv[u][1][h];
          const uint32_t f0[4] = {a.x, b.x, a.y, b.y}, f1[4] = {a.z, b.z, a.w, b.w};
          mma_16832(d, f0, x8[h][0], x8[h][1], p.w_fmt);
          mma_16832(d, f1, x8[h][2], x8[h][3], p.w_fmt);
        }
        // scales of the rows of x that are this lane's columns of d
        const float s0 = __shfl_sync(0xFFFFFFFFu, scale, int(t) * 8);
        const float s1 = __shfl_sync(0xFFFFFFFFu, scale, int(t) * 8 + 4);
        acc[mt][0] += d[0] * (ws[u][0] * s0);
        acc[mt][1] += d[1] * (ws[u][0] * s1);
        acc[mt][2] += d[2] * (ws[u][1] * s0);
        acc[mt][3] += d[3] * (ws[u][1] * s1);
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    red[warp][mt][2 * t][g] = acc[mt][0];
    red[warp][mt][2 * t + 1][g] = acc[mt][1];
    red[warp][mt][2 * t][g + 8] = acc[mt][2];
    red[warp][mt][2 * t + 1][g + 8] = acc[mt][3];
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < uint32_t(MT) * 8 * kWRows; i += kRowsWarps * 32) {
    const uint32_t n = i % kWRows, m = i / kWRows;
    if (int(m) >= p.M || n0 + int(n) >= p.N) continue;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < kRowsWarps; ++j) v += red[j][m / 8][m % 8][n];
    const int64_t at = int64_t(m) * p.ldy + n0 + n;
    if (p.y_dtype == SWZ_F32) static_cast<float*>(p.y)[at] = v;
    else if (p.y_dtype == SWZ_BF16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p.y)[at] = __float2half_rn(v);
  }
}

// largest M of the few-row kernel
constexpr int kRowsMax = 16;

template <typename T>
static int launch_rows(const RowsArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(a.N) + kWRows - 1) / kWRows));
  cfg.blockDim = dim3(kRowsWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.M <= 8) SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, linear_rows_kernel<T, 1>, a));
  else SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, linear_rows_kernel<T, 2>, a));
  return SWZ_OK;
}

// workspace: 8-bit x with rows of a multiple of 16 bytes, then its scales
static void workspace_split(int M, int K, int64_t* ldq, uint64_t* q_bytes, uint64_t* total) {
  *ldq = (int64_t(K) + 15) / 16 * 16;
  *q_bytes = (uint64_t(M) * uint64_t(*ldq) + 255u) & ~uint64_t(255);
  *total = *q_bytes + (uint64_t(K) + 127) / 128 * uint64_t(M) * 4;
}

}  // namespace f8
}  // namespace swz

using namespace swz;

extern "C" int swz_linear_fp8_workspace_size(int M, int N, int K, uint64_t* h_bytes) {
  if (!h_bytes || M < 0 || N < 0 || K < 0) return SWZ_EINVAL;
  *h_bytes = 0;
  if (M <= f8::kRowsMax || N == 0 || K == 0) return SWZ_OK;
  int64_t ldq;
  uint64_t q_bytes;
  f8::workspace_split(M, K, &ldq, &q_bytes, h_bytes);
  return SWZ_OK;
}

extern "C" int swz_linear_fp8(const void* x, int dtype, int64_t ldx, const swz_fp8_matrix* W,
                              void* y, int64_t ldy, int y_dtype, int M, int N, int K,
                              void* d_workspace, uint64_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !W) return SWZ_EINVAL;
  for (int d : {dtype, y_dtype})
    if (d != SWZ_F16 && d != SWZ_BF16 && d != SWZ_F32) return SWZ_EINVAL;
  if (W->fmt != SWZ_E4M3 && W->fmt != SWZ_E5M2) return SWZ_EINVAL;
  if (W->block != SWZ_BLOCK_ROW && W->block != SWZ_BLOCK_SQUARE) return SWZ_EINVAL;
  if (M == 0 || N == 0) return SWZ_OK;
  const int64_t es = dtype == SWZ_F32 ? 4 : 2, ys = y_dtype == SWZ_F32 ? 4 : 2;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x);
  if (!y || reinterpret_cast<uintptr_t>(y) % uintptr_t(ys) != 0 || (M > 1 && ldy < N))
    return SWZ_EINVAL;
  const int64_t kb = (int64_t(K) + 127) / 128;
  if (K > 0 && (!x || xa % uintptr_t(es) != 0 || (M > 1 && ldx < K) || !W->data ||
                !aligned16(W->data) || W->ld < K || W->ld % 16 != 0 || !W->scales ||
                !aligned4(W->scales) ||
                W->ld_scales < (W->block == SWZ_BLOCK_SQUARE ? kb : int64_t(N))))
    return SWZ_EINVAL;
  int64_t ldq;
  uint64_t q_bytes, total;
  f8::workspace_split(M, K, &ldq, &q_bytes, &total);
  const bool rows = M <= f8::kRowsMax;
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  if (K > 0 && !rows && (!ws || !aligned16(ws) || workspace_bytes < total)) return SWZ_EINVAL;
  DeviceInfo dev{};
  const int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  if (K == 0 || !rows) {
    swz_fp8_matrix a = {};
    a.data = ws;
    a.ld = ldq;
    a.scales = reinterpret_cast<float*>(ws + q_bytes);
    a.ld_scales = M;
    a.fmt = SWZ_E4M3;
    a.block = SWZ_BLOCK_ROW;
    if (K > 0) {
      const int rq = swz_quantize_fp8(x, dtype, ldx, M, K, SWZ_BLOCK_ROW, SWZ_E4M3, ws, ldq,
                                      reinterpret_cast<float*>(ws + q_bytes), M, nullptr, 0,
                                      nullptr, 0, stream);
      if (rq != SWZ_OK) return rq;
    }
    return swz_gemm_fp8(&a, W, y, ldy, y_dtype, M, N, K, nullptr, stream);
  }
  f8::RowsArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.ldx = M > 1 ? ldx : K;
  a.wide = xa % 16 == 0 && (M == 1 || (a.ldx * es) % 16 == 0);
  a.w = static_cast<const uint8_t*>(W->data);
  a.ldw = W->ld;
  a.sw = W->scales;
  a.ldsw = W->ld_scales;
  a.w_square = W->block == SWZ_BLOCK_SQUARE;
  a.w_fmt = W->fmt;
  a.y = y;
  a.ldy = M > 1 ? ldy : N;
  a.y_dtype = y_dtype;
  a.M = M;
  a.N = N;
  a.K = K;
  a.num_kb = int(kb);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SWZ_BF16) return f8::launch_rows<f8::Bf16>(a, s);
  if (dtype == SWZ_F16) return f8::launch_rows<f8::F16>(a, s);
  return f8::launch_rows<f8::F32>(a, s);
}
