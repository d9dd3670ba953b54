// layer_norm.cu -- the layer norm of rows of N values:
//     mean = sum x / N,  var = sum (x - mean)^2 / N,  rstd = 1 / sqrt(var + eps)
//     y = (x - mean) rstd w + b
// All in fp32, y rounded once.  The variance is taken of the differences from the
// mean, not as a difference of sums, so a row far from zero loses nothing.
//
// Bound: memory, x read and y written once.  A row stays in registers: TPR threads
// (a warp, or a CTA) hold NC chunks of eight values each; rows longer than 16384
// are read three times, the later times mostly from L2.
#include "layer_norm.cuh"
#include "ptx.cuh"

namespace swz {
namespace norm {

struct FwdArgs {
  rows::Span x;
  int M, N;
  Vec w, b;
  float eps;
  uint8_t* y;
  int64_t ldy;  // bytes
  int y_dtype, y_wide;
  float *mean, *rstd;
};

// TPR threads a row (32: each warp a row of its own), NC chunks a thread; NC = 0:
// any length, in loops.
template <typename T, int TPR, int NC>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR) layer_norm_kernel(const FwdArgs p) {
  constexpr int RPC = TPR == 32 ? 8 : 1;  // rows a CTA
  __shared__ float part[2][TPR / 32];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t t = threadIdx.x % TPR;
  const int64_t row = int64_t(blockIdx.x) * RPC + threadIdx.x / TPR;
  if (TPR == 32 && row >= p.M) return;  // a whole warp
  const uint8_t* x = p.x.base + row * p.x.ld;
  uint8_t* y = p.y + row * p.ldy;
  const int es = p.y_dtype == SWZ_F32 ? 4 : 2;
  const float inv = 1.0f / float(p.N);
  uint32_t w[NC ? NC : 1][T::kWords];
  // chunks of the row, rounded up so that a warp's lanes stay together
  const int64_t turns = (p.N + int64_t(TPR) * 8 - 1) / (int64_t(TPR) * 8);

  float s[1] = {0.0f};
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t k = (int64_t(c) * TPR + t) * 8;
      rows::load8<T>(x + k * T::kBytes, p.N - k, p.x, w[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += T::value(w[c], i);
  } else {
    for (int64_t c = 0; c < turns; ++c) {
      const int64_t k = (c * TPR + t) * 8;
      rows::load8<T>(x + k * T::kBytes, p.N - k, p.x, w[0]);
      float u = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) u += T::value(w[0], i);
      s[0] += u;
    }
  }
  rows::row_sums<TPR, 1>(s, part[0]);
  const float mean = s[0] * inv;

  s[0] = 0.0f;
  auto squares = [&](const uint32_t* v, int64_t k) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = T::value(v, i) - mean;
      u += k + i < p.N ? d * d : 0.0f;
    }
    s[0] += u;
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) squares(w[c], (int64_t(c) * TPR + t) * 8);
  } else {
    for (int64_t c = 0; c < turns; ++c) {
      const int64_t k = (c * TPR + t) * 8;
      rows::load8<T>(x + k * T::kBytes, p.N - k, p.x, w[0]);
      squares(w[0], k);
    }
  }
  rows::row_sums<TPR, 1>(s, part[1]);
  const float rstd = 1.0f / sqrtf(s[0] * inv + p.eps);
  if (t == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }

  auto put = [&](const uint32_t* v, int64_t k) {
    float g[8], b[8], o[8];
    load_vec(p.w, k, p.N, 1.0f, g);
    load_vec(p.b, k, p.N, 0.0f, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (T::value(v, i) - mean) * rstd * g[i] + b[i];
    rows::store8(y + k * es, p.N - k, o, p.y_dtype, p.y_wide != 0);
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) put(w[c], (int64_t(c) * TPR + t) * 8);
  } else {
    for (int64_t c = 0; c < turns; ++c) {
      const int64_t k = (c * TPR + t) * 8;
      rows::load8<T>(x + k * T::kBytes, p.N - k, p.x, w[0]);
      put(w[0], k);
    }
  }
}

template <typename T, int TPR, int NC>
static int start(const FwdArgs& a, cudaStream_t s) {
  return launch(layer_norm_kernel<T, TPR, NC>, TPR == 32 ? (uint32_t(a.M) + 7) / 8 : uint32_t(a.M),
                TPR == 32 ? 256 : TPR, a, s);
}

template <typename T>
static int dispatch(const FwdArgs& a, cudaStream_t s) {
  if (a.N <= 256) return start<T, 32, 1>(a, s);
  if (a.N <= 1024) return start<T, 32, 4>(a, s);
  if (a.N <= 4096) return start<T, 128, 4>(a, s);
  if (a.N <= 16384) return start<T, 512, 4>(a, s);
  return start<T, 512, 0>(a, s);
}

}  // namespace norm
}  // namespace swz

using namespace swz;
using namespace swz::norm;

extern "C" int swz_layer_norm(const void* x, int dtype, int64_t ldx, const void* weight,
                              int w_dtype, const void* bias, int b_dtype, double eps, void* y,
                              int y_dtype, int64_t ldy, float* mean, float* rstd, int M, int N,
                              void* stream) {
  if (M < 0 || N < 0 || !(eps >= 0.0) || eps > 3e38) return SWZ_EINVAL;
  for (int d : {dtype, w_dtype, b_dtype, y_dtype})
    if (!float_type(d)) return SWZ_EINVAL;
  if (M == 0 || N == 0) return SWZ_OK;
  if (!matrix_ok(x, dtype, ldx, M, N) || !matrix_ok(y, y_dtype, ldy, M, N)) return SWZ_EINVAL;
  if (!vector_ok(weight, w_dtype) || !vector_ok(bias, b_dtype)) return SWZ_EINVAL;
  if (!mean || !aligned4(mean) || !rstd || !aligned4(rstd)) return SWZ_EINVAL;
  DeviceInfo dev{};
  const int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  FwdArgs a{};
  a.x = rows::span_of(x, dtype, ldx, M, N);
  a.M = M;
  a.N = N;
  a.w = vec(weight, w_dtype);
  a.b = vec(bias, b_dtype);
  a.eps = float(eps);
  a.y = static_cast<uint8_t*>(y);
  a.ldy = (M > 1 ? ldy : int64_t(N)) * size_of(y_dtype);
  a.y_dtype = y_dtype;
  a.y_wide = aligned16(y) && a.ldy % 16 == 0;
  a.mean = mean;
  a.rstd = rstd;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SWZ_BF16) return dispatch<rows::Bf16>(a, s);
  if (dtype == SWZ_F16) return dispatch<rows::F16>(a, s);
  return dispatch<rows::F32>(a, s);
}
