// quantize_int8.cu -- 8-bit integers with one scale for each row of x (M x K): a
// token's activations, or an output channel's weights.  For a row with largest
// magnitude amax:
//     ac = max(amax, 2^-96),  r = 127 / ac,  scale = ac / 127   (fp32)
//     q = x r, the exact product, rounded to the nearest whole number, ties to even
// The product and the rounding are one fused multiply-add: x r + 1.5 2^23 has its
// units in the last place of fp32, so the sum's own rounding is the only one and
// its low byte is q in two's complement.  A row that holds an infinity or NaN gets
// the scale NaN and zeros, so that what is made of it is NaN.
//
// Bound: memory.  A row stays in registers between its maximum and its rounding:
// TPR threads (a warp, or a CTA) hold NC chunks of eight values each; rows longer
// than 16384 are read twice, the second time mostly from L2.
//
// Measured: 8192 x 4096 bf16 16.4 us, 6.1 TB/s of what is read and written (the copy
// bandwidth is 6.8); 77 x 1000 fp32 1.9.
#include <type_traits>

#include "common.h"
#include "int8.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace swz {
namespace i8 {

struct QuantArgs {
  rows::Span x;
  int M, K;
  uint8_t* q;
  int64_t ldq;  // bytes
  float* s;
};

// TPR threads a row (32: each warp a row of its own), NC chunks a thread; NC = 0:
// any length, in a loop, the row read again for the rounding.
template <typename T, int TPR, int NC, bool HALF>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR) quantize_int8_kernel(const QuantArgs p) {
  constexpr int RPC = TPR == 32 ? 8 : 1;  // rows a CTA
  constexpr int QB = HALF ? 2 : 1;
  __shared__ uint32_t part[TPR / 32];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t t = threadIdx.x % TPR;
  const int64_t row = int64_t(blockIdx.x) * RPC + threadIdx.x / TPR;
  if (TPR == 32 && row >= p.M) return;  // a whole warp
  const uint8_t* x = p.x.base + row * p.x.ld;
  uint32_t w[NC ? NC : 1][T::kWords];
  uint32_t m = 0;
  const int64_t chunks = (int64_t(p.K) + 7) / 8;
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t k = (int64_t(c) * TPR + t) * 8;
      rows::load8<T>(x + k * T::kBytes, p.K - k, p.x, w[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) m = max(m, chunk_max<T>(w[c]));
  } else {
    for (int64_t c = t; c < chunks; c += TPR) {
      rows::load8<T>(x + c * 8 * T::kBytes, p.K - c * 8, p.x, w[0]);
      m = max(m, chunk_max<T>(w[0]));
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if constexpr (TPR > 32) {
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) m = max(m, part[i]);
  }
  float r, scale;
  const bool bad = row_scale(T::max_bits(m), r, scale);
  if (t == 0) p.s[row] = scale;
  uint8_t* q = p.q + row * p.ldq;
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t k = (int64_t(c) * TPR + t) * 8;
      if (k < p.K) store_q<T, HALF>(q + k * QB, p.K - k, w[c], r, bad);
    }
  } else {
    for (int64_t c = t; c < chunks; c += TPR) {
      rows::load8<T>(x + c * 8 * T::kBytes, p.K - c * 8, p.x, w[0]);
      store_q<T, HALF>(q + c * 8 * QB, p.K - c * 8, w[0], r, bad);
    }
  }
}

template <typename T, int TPR, int NC>
static int launch(const QuantArgs& a, bool half, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(TPR == 32 ? (uint32_t(a.M) + 7) / 8 : uint32_t(a.M));
  cfg.blockDim = dim3(TPR == 32 ? 256 : TPR);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (half) SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, quantize_int8_kernel<T, TPR, NC, true>, a));
  else SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, quantize_int8_kernel<T, TPR, NC, false>, a));
  return SWZ_OK;
}

template <typename T>
static int dispatch(const QuantArgs& a, bool half, cudaStream_t s) {
  if (a.K <= 256) return launch<T, 32, 1>(a, half, s);
  if (a.K <= 1024) return launch<T, 32, 4>(a, half, s);
  if (a.K <= 4096) return launch<T, 128, 4>(a, half, s);
  if (a.K <= 16384) return launch<T, 512, 4>(a, half, s);
  return launch<T, 512, 0>(a, half, s);
}

int quantize_rows(const void* x, int dtype, int64_t ldx, int M, int K, void* q, int64_t ldq,
                  float* scales, bool half, cudaStream_t s) {
  QuantArgs a{};
  a.x = rows::span_of(x, dtype, ldx, M, K);
  a.M = M;
  a.K = K;
  a.q = static_cast<uint8_t*>(q);
  a.ldq = ldq;
  a.s = scales;
  if (dtype == SWZ_BF16) return dispatch<rows::Bf16>(a, half, s);
  if (dtype == SWZ_F16) return dispatch<rows::F16>(a, half, s);
  return dispatch<rows::F32>(a, half, s);
}

}  // namespace i8
}  // namespace swz

using namespace swz;

extern "C" int swz_quantize_int8(const void* x, int dtype, int64_t ldx, int M, int K, void* q,
                                 int64_t ldq, float* scales, void* stream) {
  if (M < 0 || K < 0) return SWZ_EINVAL;
  if (dtype != SWZ_F16 && dtype != SWZ_BF16 && dtype != SWZ_F32) return SWZ_EINVAL;
  if (M == 0) return SWZ_OK;
  const uintptr_t es = dtype == SWZ_F32 ? 4 : 2;
  if (!scales || !aligned4(scales)) return SWZ_EINVAL;
  if (K > 0 && (!x || reinterpret_cast<uintptr_t>(x) % es != 0 || (M > 1 && ldx < K) || !q ||
                !aligned16(q) || ldq < K || ldq % 16 != 0))
    return SWZ_EINVAL;
  const int64_t width = int64_t(K) * int64_t(es);
  const RowsInMemory input{x, M, M > 1 ? ldx * int64_t(es) : width, width};
  if (rows_meet(input, RowsInMemory{q, M, M > 1 ? ldq : K, K}) ||
      rows_meet(input, RowsInMemory{scales, 1, 0, int64_t(M) * 4}))
    return SWZ_EINVAL;
  DeviceInfo dev{};
  const int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  return i8::quantize_rows(x, dtype, ldx, M, K, q, ldq, scales, false,
                           static_cast<cudaStream_t>(stream));
}
