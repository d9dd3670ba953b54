// layer_norm_backward.cu -- the gradient of the layer norm.  With xhat = (x - mean)
// rstd and g = dy w, by rows
//     dx = rstd (g - sum g / N - xhat sum(g xhat) / N)
// and over all rows dw = sum dy xhat, db = sum dy.  All in fp32, each result rounded
// once.
//
// Bound: memory, x and dy read and dx written once.  A CTA takes every P-th row (or
// every P-th eight rows, a row a warp, where rows are short), and a thread the same
// columns of each of them, so that its parts of dw and db stay in registers; the
// P partial rows go to the workspace and a second kernel adds them in order
// (deterministic, no atomics).  The next row's loads are under way while this one's
// two sums cross the CTA.  Rows longer than 16384 take dx and the partial sums in
// two kernels that read both inputs again.
#include <type_traits>

#include "layer_norm.cuh"
#include "ptx.cuh"

namespace swz {
namespace norm {

constexpr int kMaxParts = 608;  // partial rows, whatever the device

struct BwdArgs {
  rows::Span x, dy;
  int M, N;
  Vec w;
  const float *mean, *rstd;
  uint8_t* dx;  // NULL: not wanted
  int64_t lddx;  // bytes
  int dx_dtype, dx_wide;
  float* parts;  // (P, 2, N): dw, then db; NULL: neither wanted
};

// TPR threads a row (32: each warp rows of its own), NC chunks a thread.
template <typename X, typename D, int TPR, int NC>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR)
    layer_norm_backward_kernel(const BwdArgs p) {
  constexpr int RPC = TPR == 32 ? 8 : 1;  // rows a CTA and turn
  __shared__ float part[2][2 * (TPR / 32)];
  __shared__ float both[TPR == 32 ? 2 * NC * 256 : 1];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t t = threadIdx.x % TPR;
  const int es = p.dx_dtype == SWZ_F32 ? 4 : 2;
  const float inv = 1.0f / float(p.N);

  float w[NC][8], dw[NC][8], db[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    load_vec(p.w, (int64_t(c) * TPR + t) * 8, p.N, 1.0f, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0.0f;
  }
  uint32_t xw[NC][X::kWords], dw_[NC][D::kWords];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t k = (int64_t(c) * TPR + t) * 8;
      rows::load8<X>(p.x.base + row * p.x.ld + k * X::kBytes, p.N - k, p.x, xw[c]);
      rows::load8<D>(p.dy.base + row * p.dy.ld + k * D::kBytes, p.N - k, p.dy, dw_[c]);
    }
    mean = p.mean[row];
    rstd = p.rstd[row];
  };
  const int64_t step = int64_t(gridDim.x) * RPC;
  int64_t row = int64_t(blockIdx.x) * RPC + threadIdx.x / TPR;
  if (row < p.M) fetch(row);
  for (uint32_t turn = 0; row < p.M; row += step, turn ^= 1u) {
    float xhat[NC][8], d[NC][8], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = (X::value(xw[c], i) - mean) * rstd, v = D::value(dw_[c], i);
        dw[c][i] += v * h;
        db[c][i] += v;
        xhat[c][i] = h;
        d[c][i] = v * w[c][i];
        s[0] += d[c][i];
        s[1] += d[c][i] * h;
      }
    const float rs = rstd;
    if (row + step < p.M) fetch(row + step);
    if (p.dx) {
      rows::row_sums<TPR, 2>(s, part[turn]);
      const float a = s[0] * inv, b = s[1] * inv;
      uint8_t* dx = p.dx + row * p.lddx;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int64_t k = (int64_t(c) * TPR + t) * 8;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rs * (d[c][i] - a - xhat[c][i] * b);
        rows::store8(dx + k * es, p.N - k, o, p.dx_dtype, p.dx_wide != 0);
      }
    }
  }
  if (!p.parts) return;
  if constexpr (TPR == 32) {
    // the eight warps' sums, added in order
    for (uint32_t i = 0; i < 8; ++i) {
      if (threadIdx.x / 32 == i)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* at = both + (c * 32 + t) * 8 + e;
            at[0] = i ? at[0] + dw[c][e] : dw[c][e];
            at[NC * 256] = i ? at[NC * 256] + db[c][e] : db[c][e];
          }
      __syncthreads();
    }
    float* out = p.parts + int64_t(blockIdx.x) * 2 * p.N;
    for (int k = int(threadIdx.x); k < p.N; k += 256) {
      out[k] = both[k];
      out[p.N + k] = both[NC * 256 + k];
    }
  } else {
    float* out = p.parts + int64_t(blockIdx.x) * 2 * p.N;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t k = (int64_t(c) * TPR + t) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < p.N) {
          out[k + i] = dw[c][i];
          out[p.N + k + i] = db[c][i];
        }
    }
  }
}

// ---- rows of any length -----------------------------------------------------------
template <typename X, typename D>
__global__ void __launch_bounds__(512) long_dx_kernel(const BwdArgs p) {
  constexpr int TPR = 512;
  __shared__ float part[2 * (TPR / 32)];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int es = p.dx_dtype == SWZ_F32 ? 4 : 2;
  const float inv = 1.0f / float(p.N), mean = p.mean[row], rstd = p.rstd[row];
  const int64_t turns = (int64_t(p.N) + TPR * 8 - 1) / (TPR * 8);
  uint32_t xw[X::kWords], dw[D::kWords];
  float w[8], s[2] = {0.0f, 0.0f};
  auto fetch = [&](int64_t k) {
    rows::load8<X>(p.x.base + row * p.x.ld + k * X::kBytes, p.N - k, p.x, xw);
    rows::load8<D>(p.dy.base + row * p.dy.ld + k * D::kBytes, p.N - k, p.dy, dw);
    load_vec(p.w, k, p.N, 1.0f, w);
  };
  for (int64_t c = 0; c < turns; ++c) {
    fetch((c * TPR + threadIdx.x) * 8);
    float u[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = D::value(dw, i) * w[i];
      u[0] += d;
      u[1] += d * ((X::value(xw, i) - mean) * rstd);
    }
    s[0] += u[0];
    s[1] += u[1];
  }
  rows::row_sums<TPR, 2>(s, part);
  const float a = s[0] * inv, b = s[1] * inv;
  for (int64_t c = 0; c < turns; ++c) {
    const int64_t k = (c * TPR + threadIdx.x) * 8;
    fetch(k);
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = rstd * (D::value(dw, i) * w[i] - a - (X::value(xw, i) - mean) * rstd * b);
    rows::store8(p.dx + row * p.lddx + k * es, p.N - k, o, p.dx_dtype, p.dx_wide != 0);
  }
}

// partial sums over every gridDim.y-th row, a column a thread
template <typename X, typename D>
__global__ void __launch_bounds__(256) long_parts_kernel(const BwdArgs p) {
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (k >= p.N) return;
  constexpr int XT = X::kBytes == 4 ? SWZ_F32 : std::is_same<X, rows::Bf16>::value ? SWZ_BF16 : SWZ_F16;
  constexpr int DT = D::kBytes == 4 ? SWZ_F32 : std::is_same<D, rows::Bf16>::value ? SWZ_BF16 : SWZ_F16;
  float dw = 0.0f, db = 0.0f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
    const float v = rows::load1(p.dy.base + row * p.dy.ld + k * D::kBytes, DT);
    const float x = rows::load1(p.x.base + row * p.x.ld + k * X::kBytes, XT);
    dw += v * ((x - p.mean[row]) * p.rstd[row]);
    db += v;
  }
  float* out = p.parts + int64_t(blockIdx.y) * 2 * p.N;
  out[k] = dw;
  out[p.N + k] = db;
}

// ---- the partial rows' sum ----------------------------------------------------------
struct SumArgs {
  const float* parts;
  int P, N;
  uint8_t *dw, *db;  // either may be NULL
  int dtype;
};

// blockIdx.y: 0 dw, 1 db.  32 columns a CTA, its 8 warps every eighth partial row each.
__global__ void __launch_bounds__(256) sum_parts_kernel(const SumArgs p) {
  __shared__ float part[8][32];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const int64_t k = int64_t(blockIdx.x) * 32 + threadIdx.x % 32;
  uint8_t* out = blockIdx.y ? p.db : p.dw;
  if (!out) return;
  float s = 0.0f;
  if (k < p.N) {
    const float* src = p.parts + int64_t(blockIdx.y) * p.N + k;
#pragma unroll 8
    for (int i = int(threadIdx.x / 32); i < p.P; i += 8) s += src[int64_t(i) * 2 * p.N];
  }
  part[threadIdx.x / 32][threadIdx.x % 32] = s;
  __syncthreads();
  if (threadIdx.x < 32 && k < p.N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
    rows::store1(out + k * (p.dtype == SWZ_F32 ? 4 : 2), s, p.dtype);
  }
}

template <typename X, typename D, int TPR, int NC>
static int start(const BwdArgs& a, int* P, int num_sms, cudaStream_t s) {
  auto kern = layer_norm_backward_kernel<X, D, TPR, NC>;
  constexpr int threads = TPR == 32 ? 256 : TPR;
  int resident = 0;
  SWZ_CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kern, threads, 0));
  int64_t grid = (int64_t(a.M) + (TPR == 32 ? 7 : 0)) / (TPR == 32 ? 8 : 1);
  const int64_t cap = int64_t(num_sms) * (resident < 1 ? 1 : resident);
  if (grid > cap) grid = cap;
  if (a.parts && grid > kMaxParts) grid = kMaxParts;
  *P = int(grid);
  return launch(kern, uint32_t(grid), threads, a, s);
}

template <typename X, typename D>
static int dispatch(const BwdArgs& a, int* P, int num_sms, cudaStream_t s) {
  if (a.N <= 256) return start<X, D, 32, 1>(a, P, num_sms, s);
  if (a.N <= 1024) return start<X, D, 32, 4>(a, P, num_sms, s);
  if (a.N <= 2048) return start<X, D, 128, 2>(a, P, num_sms, s);
  if (a.N <= 4096) return start<X, D, 256, 2>(a, P, num_sms, s);
  if (a.N <= 8192) return start<X, D, 512, 2>(a, P, num_sms, s);
  if (a.N <= 16384) return start<X, D, 512, 4>(a, P, num_sms, s);
  if (a.dx) {
    const int rc = launch(long_dx_kernel<X, D>, uint32_t(a.M), 512, a, s);
    if (rc != SWZ_OK) return rc;
  }
  if (!a.parts) return SWZ_OK;
  *P = a.M < 64 ? a.M : 64;
  const dim3 grid(uint32_t((int64_t(a.N) + 255) / 256), uint32_t(*P));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, long_parts_kernel<X, D>, a));
  return SWZ_OK;
}

template <typename X>
static int dispatch_dy(const BwdArgs& a, int dy_dtype, int* P, int num_sms, cudaStream_t s) {
  if (dy_dtype == SWZ_BF16) return dispatch<X, rows::Bf16>(a, P, num_sms, s);
  if (dy_dtype == SWZ_F16) return dispatch<X, rows::F16>(a, P, num_sms, s);
  return dispatch<X, rows::F32>(a, P, num_sms, s);
}

}  // namespace norm
}  // namespace swz

using namespace swz;
using namespace swz::norm;

extern "C" int swz_layer_norm_backward_workspace_size(int M, int N, uint64_t* h_bytes) {
  if (!h_bytes || M < 0 || N < 0) return SWZ_EINVAL;
  *h_bytes = uint64_t(M < kMaxParts ? M : kMaxParts) * 2 * uint64_t(N) * 4;
  return SWZ_OK;
}

extern "C" int swz_layer_norm_backward(const void* dy, int dy_dtype, int64_t lddy, const void* x,
                                       int dtype, int64_t ldx, const void* weight, int w_dtype,
                                       const float* mean, const float* rstd, void* dx,
                                       int dx_dtype, int64_t lddx, void* dw, void* db,
                                       int dw_dtype, int M, int N, void* d_workspace,
                                       uint64_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0) return SWZ_EINVAL;
  for (int d : {dy_dtype, dtype, w_dtype, dx_dtype, dw_dtype})
    if (!float_type(d)) return SWZ_EINVAL;
  if (N == 0) return SWZ_OK;
  if (M > 0 && !dx && !dw && !db) return SWZ_EINVAL;
  if (!vector_ok(weight, w_dtype) || !vector_ok(dw, dw_dtype) || !vector_ok(db, dw_dtype))
    return SWZ_EINVAL;
  const bool sums = dw || db;
  if (M > 0) {
    if (!matrix_ok(dy, dy_dtype, lddy, M, N) || !matrix_ok(x, dtype, ldx, M, N) ||
        (dx && !matrix_ok(dx, dx_dtype, lddx, M, N)))
      return SWZ_EINVAL;
    if (!mean || !aligned4(mean) || !rstd || !aligned4(rstd)) return SWZ_EINVAL;
    uint64_t need = 0;
    swz_layer_norm_backward_workspace_size(M, N, &need);
    if (sums && (!d_workspace || !aligned16(d_workspace) || workspace_bytes < need))
      return SWZ_EINVAL;
  }
  DeviceInfo dev{};
  int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {  // the sum over no rows
    const size_t bytes = size_t(N) * size_t(size_of(dw_dtype));
    if (dw) SWZ_CUDA_TRY(cudaMemsetAsync(dw, 0, bytes, s));
    if (db) SWZ_CUDA_TRY(cudaMemsetAsync(db, 0, bytes, s));
    return SWZ_OK;
  }
  BwdArgs a{};
  a.x = rows::span_of(x, dtype, ldx, M, N);
  a.dy = rows::span_of(dy, dy_dtype, lddy, M, N);
  a.M = M;
  a.N = N;
  a.w = vec(weight, w_dtype);
  a.mean = mean;
  a.rstd = rstd;
  a.dx = static_cast<uint8_t*>(dx);
  a.lddx = (M > 1 ? lddx : int64_t(N)) * size_of(dx_dtype);
  a.dx_dtype = dx_dtype;
  a.dx_wide = aligned16(dx) && a.lddx % 16 == 0;
  a.parts = sums ? static_cast<float*>(d_workspace) : nullptr;
  int P = 0;
  if (dtype == SWZ_BF16) rc = dispatch_dy<rows::Bf16>(a, dy_dtype, &P, dev.num_sms, s);
  else if (dtype == SWZ_F16) rc = dispatch_dy<rows::F16>(a, dy_dtype, &P, dev.num_sms, s);
  else rc = dispatch_dy<rows::F32>(a, dy_dtype, &P, dev.num_sms, s);
  if (rc != SWZ_OK || !sums) return rc;
  SumArgs g{};
  g.parts = a.parts;
  g.P = P;
  g.N = N;
  g.dw = static_cast<uint8_t*>(dw);
  g.db = static_cast<uint8_t*>(db);
  g.dtype = dw_dtype;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(uint32_t((int64_t(N) + 31) / 32), 2);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, sum_parts_kernel, g));
  return SWZ_OK;
}
