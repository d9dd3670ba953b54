// layer_norm_backward.cu -- the gradient of the layer norm.  With xhat = (x - mean)
// rstd and g = dy w, by rows
//     dx = rstd (g - sum g / N - xhat sum(g xhat) / N)
// and over all rows dw = sum dy xhat, db = sum dy.  All in fp32, each result rounded
// once.
//
// Bound: memory, x and dy read and dx written once.  A CTA takes every P-th row (or
// every P-th eight rows, a row a warp, where rows have 512 values or less), and a
// thread the same columns of each of them, so that its parts of dw and db stay in
// registers; the P partial rows go to the workspace and a second kernel adds them in
// order (deterministic, no atomics).  The next row's loads are under way while this
// one's two sums cross the CTA; w comes from L1, where x and dy leave it alone.  As many
// threads as the row asks for, each with NC chunks of eight columns.  P is a quarter of
// the rows at most, or one an SM, since a partial row is 16 bytes a column, written and
// read, and a row of bf16 inputs and result 6.  Rows longer than 16384 take the partial
// sums and dx in two kernels that both read the inputs.
//
// Measured: 8192 x 4096 bf16 41.3 us (29.7 at the copy bandwidth; 35 without dw and db),
// fp32 68.5 (59.4), 16384 x 1000 bf16 26.9 (14.5), 4096 x 10240 92 (37, four chunks a
// thread), 1001 x 600 fp32 7.8 (1.1), 1001 x 1999 fp16 22 (1.8).  With three CTAs an SM
// instead of two and a row's values worked out twice for it 52 us; an element an
// instruction 45.
#include <algorithm>
#include <type_traits>

#include "layer_norm.cuh"
#include "ptx.cuh"

namespace swz {
namespace norm {

constexpr int kMaxParts = 608;  // partial rows, whatever the device
static int64_t pitch_of(int N) { return (int64_t(N) + 7) / 8 * 8; }

struct BwdArgs {
  rows::Span x, dy;
  int M, N;
  Vec w;
  const float *mean, *rstd;
  uint8_t* dx;  // NULL: not wanted
  int64_t lddx;  // bytes
  int dx_dtype, dx_wide;
  float* parts;  // (P, 2, pitch): dw, then db; NULL: neither wanted
  int64_t pitch;
};

// Whether mean rstd leaves fp32's range.  Beyond a row's end x reads as zero, and its xhat
// there, -mean rstd, times the zero of dy makes the sum of g xhat NaN.  That sum is zero in
// truth: a row with a value other than its mean has rstd <= sqrt(N) / |x - mean| <= 2^40 /
// |mean|, so every value of such a row is its mean (1e33 throughout, with an eps of 1e-12).
__device__ __forceinline__ bool far_constant(float mean, float rstd) {
  return isinf(mean * rstd) && isfinite(mean) && isfinite(rstd);
}

// NC chunks a thread; WARP: a row a warp, eight a CTA, otherwise a row the CTA; G: the
// common case (layer_norm.cuh) or 0.
template <typename X, typename D, int NC, bool WARP, int G>
__global__ void __launch_bounds__(WARP ? 256 : 512) layer_norm_backward_kernel(const BwdArgs p) {
  __shared__ float2 part[2][16];
  __shared__ ulonglong2 sums[WARP ? NC * 128 : 1];  // of the warps: dw, then db
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int width = WARP ? 32 : int(blockDim.x), warps = WARP ? 1 : int(blockDim.x) / 32;
  const int t = WARP ? int(lane) : int(threadIdx.x);
  const int es = p.dx_dtype == SWZ_F32 ? 4 : 2;
  const float inv = 1.0f / float(p.N);

  uint64_t dw[NC][4], db[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[c][i] = db[c][i] = 0ull;
  uint32_t xw[NC][X::kWords], dyw[NC][D::kWords];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t row) {
    const uint8_t *x = p.x.base + row * p.x.ld, *dy = p.dy.base + row * p.dy.ld;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (c * width + t) * 8;
      if constexpr (G) {
        fast_load<X>(x + int64_t(k) * X::kBytes, k < p.N, xw[c]);
        fast_load<D>(dy + int64_t(k) * D::kBytes, k < p.N, dyw[c]);
      } else {
        rows::load8_once<X>(x + int64_t(k) * X::kBytes, p.N - k, p.x, xw[c]);
        rows::load8_once<D>(dy + int64_t(k) * D::kBytes, p.N - k, p.dy, dyw[c]);
      }
    }
    mean = p.mean[row];
    rstd = p.rstd[row];
  };
  // With four chunks a thread there are no registers for a row's values beside the next
  // one's: they are worked out again from the inputs as they were loaded.
  constexpr bool AHEAD = NC <= 2;
  const int64_t step = int64_t(gridDim.x) * (WARP ? 8 : 1);
  int64_t row = WARP ? int64_t(blockIdx.x) * 8 + warp : int64_t(blockIdx.x);
  if (AHEAD && row < p.M) fetch(row);
  for (uint32_t turn = 0; row < p.M; row += step, turn ^= 1u) {
    if (!AHEAD) fetch(row);
    uint64_t xhat[AHEAD ? NC : 1][4], d[AHEAD ? NC : 1][4], s0 = 0ull, s1 = 0ull;
    const uint64_t m2 = both(-mean), r2 = both(rstd);
    const bool far = far_constant(mean, rstd);
    auto values = [&](int c, uint64_t (&h)[4], uint64_t (&g)[4], uint64_t (&v)[4]) {
      uint64_t x[4], w[4];
      pairs_of<X>(xw[c], x);
      pairs_of<D>(dyw[c], v);
      const int k = (c * width + t) * 8;
      // (beyond the row dy is zero, and so is what it is multiplied by)
      if constexpr (G) fast_vec<X, G>(p.w.p, k < p.N ? k : 0, w);
      else load_vec2(p.w, k, p.N, 1.0f, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = pipe::mul2(add2(x[i], m2), r2);
        g[i] = pipe::mul2(v[i], w[i]);
      }
    };
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      uint64_t(&h)[4] = xhat[AHEAD ? c : 0];
      uint64_t(&g)[4] = d[AHEAD ? c : 0];
      uint64_t v[4];
      values(c, h, g, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw[c][i] = pipe::fma2(v[i], h[i], dw[c][i]);
        db[c][i] = add2(db[c][i], v[i]);
        s0 = add2(s0, g[i]);
        s1 = pipe::fma2(g[i], h[i], s1);
      }
    }
    if (AHEAD && row + step < p.M) fetch(row + step);
    if (p.dx) {
      float a = rows::warp_sum(sum_of(s0)), b = rows::warp_sum(sum_of(s1));
      if constexpr (!WARP) {
        if (lane == 0) part[turn][warp] = make_float2(a, b);
        __syncthreads();
        a = b = 0.0f;
        for (int i = 0; i < warps; ++i) {
          const float2 u = part[turn][i];
          a += u.x;
          b += u.y;
        }
      }
      const uint64_t a2 = both(-a * inv), b2 = both(far ? 0.0f : -b * inv);
      uint8_t* dx = p.dx + row * p.lddx;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int k = (c * width + t) * 8;
        uint64_t(&h)[4] = xhat[AHEAD ? c : 0];
        uint64_t(&g)[4] = d[AHEAD ? c : 0];
        uint64_t o[4];
        if (!AHEAD) values(c, h, g, o);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = pipe::mul2(pipe::fma2(h[i], b2, add2(g[i], a2)), r2);
        if constexpr (G) {
          if (k < p.N) fast_store<X>(dx + int64_t(k) * X::kBytes, o);
        } else {
          store_pairs(dx + int64_t(k) * es, p.N - k, o, p.dx_dtype, p.dx_wide != 0);
        }
      }
    }
  }
  if (!p.parts) return;
  // partial rows of `pitch` values, a multiple of eight: whole chunks are stored
  float* const out = p.parts + int64_t(blockIdx.x) * 2 * p.pitch;
  auto put = [&](int k, int e, ulonglong2 v) {  // e: two quads of dw, then of db
    *reinterpret_cast<ulonglong2*>(out + (e < 2 ? 0 : p.pitch) + k + 4 * (e & 1)) = v;
  };
  if constexpr (WARP) {
    // the eight warps' sums, added in order
    for (uint32_t i = 0; i < 8; ++i) {
      if (warp == i)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t* v = e < 2 ? &dw[c][2 * e] : &db[c][2 * e - 4];
            ulonglong2& at = sums[(c * 4 + e) * 32 + lane];
            at = i ? make_ulonglong2(add2(at.x, v[0]), add2(at.y, v[1])) : make_ulonglong2(v[0], v[1]);
          }
      __syncthreads();
    }
    if (warp == 0)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int k = (c * 32 + int(lane)) * 8;
        if (k < p.N)
#pragma unroll
          for (int e = 0; e < 4; ++e) put(k, e, sums[(c * 4 + e) * 32 + lane]);
      }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (c * width + t) * 8;
      if (k < p.N)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t* v = e < 2 ? &dw[c][2 * e] : &db[c][2 * e - 4];
          put(k, e, make_ulonglong2(v[0], v[1]));
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
  const float a = s[0] * inv, b = far_constant(mean, rstd) ? 0.0f : s[1] * inv;
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
  float* out = p.parts + int64_t(blockIdx.y) * 2 * p.pitch;
  out[k] = dw;
  out[p.pitch + k] = db;
}

// ---- the partial rows' sum ----------------------------------------------------------
struct SumArgs {
  const float* parts;
  int P, N;
  int64_t pitch;
  uint8_t *dw, *db;  // either may be NULL
  int dtype;
};

// blockIdx.y: 0 dw, 1 db.  32 columns a CTA; a warp adds every 32nd partial row, so
// that a few loads a thread, all in flight, do it.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const SumArgs p) {
  __shared__ float part[32][32];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t k = int64_t(blockIdx.x) * 32 + lane;
  uint8_t* out = blockIdx.y ? p.db : p.dw;
  if (!out) return;
  float s = 0.0f;
  if (k < p.N) {
    const float* src = p.parts + int64_t(blockIdx.y) * p.pitch + k;
#pragma unroll 8
    for (int i = int(warp); i < p.P; i += 32) s += src[int64_t(i) * 2 * p.pitch];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && k < p.N) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += part[i][lane];
    rows::store1(out + k * (p.dtype == SWZ_F32 ? 4 : 2), s, p.dtype);
  }
}

template <typename X, typename D, int NC, bool WARP, int G>
static int start_kind(const BwdArgs& a, int* P, int num_sms, cudaStream_t s) {
  const int threads = WARP ? 256 : threads_of(a.N, NC);
  int resident = 0;
  const int rc = resident_ctas<layer_norm_backward_kernel<X, D, NC, WARP, G>>(threads, &resident);
  if (rc != SWZ_OK) return rc;
  const int64_t rows = WARP ? (int64_t(a.M) + 7) / 8 : int64_t(a.M);
  int64_t most = int64_t(num_sms) * resident;
  if (a.parts) {
    const int64_t few = std::max(int64_t(num_sms), rows / 4);
    most = std::min(std::min(most, few), int64_t(kMaxParts));
  }
  *P = int(std::min(rows, most));
  return launch(layer_norm_backward_kernel<X, D, NC, WARP, G>, uint32_t(*P), uint32_t(threads), a, s);
}

template <typename X, typename D, int NC, bool WARP>
static int start(const BwdArgs& a, int* P, int num_sms, cudaStream_t s) {
  const int g = kind_of<X>(a.w);
  if (g == 0 || !a.x.wide || !a.dy.wide || a.N % 8 != 0 ||
      (a.dx && (!a.dx_wide || a.dx_dtype != code_of<X>())))
    return start_kind<X, D, NC, WARP, 0>(a, P, num_sms, s);
  if constexpr (X::kBytes == 2)
    if (g == 2) return start_kind<X, D, NC, WARP, 2>(a, P, num_sms, s);
  return start_kind<X, D, NC, WARP, 1>(a, P, num_sms, s);
}

template <typename X, typename D>
static int dispatch(const BwdArgs& a, int* P, int num_sms, cudaStream_t s) {
  if (a.N <= 256) return start<X, D, 1, true>(a, P, num_sms, s);
  if (a.N <= 512) return start<X, D, 2, true>(a, P, num_sms, s);
  if (a.N <= 8192) return start<X, D, 2, false>(a, P, num_sms, s);
  if (a.N <= 16384) return start<X, D, 4, false>(a, P, num_sms, s);
  if (a.parts) {  // first: dx may lie over x or dy
    *P = a.M < 64 ? a.M : 64;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(uint32_t((int64_t(a.N) + 255) / 256), uint32_t(*P));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, long_parts_kernel<X, D>, a));
  }
  return a.dx ? launch(long_dx_kernel<X, D>, uint32_t(a.M), 512, a, s) : int(SWZ_OK);
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
  *h_bytes = uint64_t(M < kMaxParts ? M : kMaxParts) * 2 * uint64_t(pitch_of(N)) * 4;
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
    if (dx) {
      const RowsInMemory result = rows_at(dx, dx_dtype, lddx, M, N);
      if (!may_lie(result, dx_dtype, rows_at(x, dtype, ldx, M, N), dtype) ||
          !may_lie(result, dx_dtype, rows_at(dy, dy_dtype, lddy, M, N), dy_dtype) ||
          !apart(result, weight, N * size_of(w_dtype)) || !apart(result, mean, int64_t(M) * 4) ||
          !apart(result, rstd, int64_t(M) * 4))
        return SWZ_EINVAL;
    }
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
  a.pitch = pitch_of(N);
  int P = 0;
  if (dtype == SWZ_BF16) rc = dispatch_dy<rows::Bf16>(a, dy_dtype, &P, dev.num_sms, s);
  else if (dtype == SWZ_F16) rc = dispatch_dy<rows::F16>(a, dy_dtype, &P, dev.num_sms, s);
  else rc = dispatch_dy<rows::F32>(a, dy_dtype, &P, dev.num_sms, s);
  if (rc != SWZ_OK || !sums) return rc;
  SumArgs g{};
  g.parts = a.parts;
  g.P = P;
  g.N = N;
  g.pitch = a.pitch;
  g.dw = static_cast<uint8_t*>(dw);
  g.db = static_cast<uint8_t*>(db);
  g.dtype = dw_dtype;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(uint32_t((int64_t(N) + 31) / 32), 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, sum_parts_kernel, g));
  return SWZ_OK;
}
