// layer_norm.cu -- the layer norm of rows of N values:
//     mean = sum x / N,  var = sum (x - mean)^2 / N,  rstd = 1 / sqrt(var + eps)
//     y = (x - mean) rstd w + b
// All in fp32, y rounded once.  The variance is taken of differences from a mean, not
// as a difference of sums, so that of a row far from zero loses nothing: each warp takes
// the mean of its part of the row and the squares around that, and the parts are joined by
//     sum (x - mean)^2 = sum over the warps of  M2_w + n_w (mean_w - mean)^2
// which needs one exchange between the warps instead of two.  The mean itself is a sum of
// fp32 additions, up to 4 units in its last place off (rows of up to 20000 values, measured),
// and y as much times rstd w: up to 0.27 for constant rows of 500 to 2000 with an eps of
// 1e-5, of which the rounding of a mean to fp32 alone may cost 0.04.  A mean corrected by
// the sum of x - mean was exact there, and took 29.2 us instead of 25.9 for 8192 x 4096 bf16.
//
// Bound: memory, x read and y written once.  A row stays in registers: the threads of a
// CTA (a warp where rows have 512 values or less) hold NC chunks of eight values each,
// as many threads as the row asks for.  CTAs stay and take one row after another, the
// next row's loads under way while this one is worked on; w and b stay in registers
// where they fit (two chunks a thread, the common case of layer_norm.cuh) and come from
// L1, where x leaves them alone, otherwise.  Rows longer than 16384 are read three
// times, the later times mostly from L2.
//
// Measured: 8192 x 4096 bf16 26.3 us (5.1 TB/s of what is read and written; 19.8 at the
// copy bandwidth), fp32 47.9 (39.6), 16384 x 2048 bf16 22.5 (19.8), 16384 x 1000 11.7
// (9.7), 4096 x 10240 44 (24.7, four chunks), 1001 x 1999 fp16, whose rows start
// anywhere, 8.5 (1.2).  Of 8192 x 4096: with w and b from L1 31.9 (the load-store unit
// 74 % busy), an element an instruction 39, two CTAs an SM instead of three 31.6, the
// next rows through a ring of bulk copies 50 (in the form with an element an
// instruction, 43 without the ring).
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

// NC chunks a thread; WARP: a row a warp, eight a CTA, otherwise a row the CTA; G: the
// common case (layer_norm.cuh) or 0; MOST: threads of a CTA, at most.
template <typename T, int NC, bool WARP, int G, int MOST>
__global__ void __launch_bounds__(MOST, WARP ? 4 : MOST == 256 ? 3 : G && NC == 2 ? 1 : 2)
    layer_norm_kernel(const FwdArgs p) {
  constexpr bool HOLD = G && NC == 2 && !WARP;  // weight and bias in registers
  __shared__ float2 part[2][16];
  __shared__ float counts[16];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int width = WARP ? 32 : int(blockDim.x), warps = WARP ? 1 : int(blockDim.x) / 32;
  const int t = WARP ? int(lane) : int(threadIdx.x);
  const int es = p.y_dtype == SWZ_F32 ? 4 : 2;
  const float inv = 1.0f / float(p.N);
  // values of the row that this warp holds
  int mine = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int left = p.N - (c * width + (t - int(lane))) * 8;
    mine += left < 0 ? 0 : left > 256 ? 256 : left;
  }
  const bool all = mine == NC * 256;
  const float inv_mine = mine ? 1.0f / float(mine) : 0.0f;
  if (!WARP && lane == 0) counts[warp] = float(mine);

  uint32_t w[NC][T::kWords];
  auto fetch = [&](int64_t row) {
    const uint8_t* x = p.x.base + row * p.x.ld;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (c * width + t) * 8;
      if constexpr (G) fast_load<T>(x + int64_t(k) * T::kBytes, k < p.N, w[c]);
      else rows::load8_once<T>(x + int64_t(k) * T::kBytes, p.N - k, p.x, w[c]);
    }
  };
  const int64_t step = int64_t(gridDim.x) * (WARP ? 8 : 1);
  int64_t row = WARP ? int64_t(blockIdx.x) * 8 + warp : int64_t(blockIdx.x);
  if (row < p.M) fetch(row);
  uint64_t held[HOLD ? 2 * NC : 1][4];
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (c * width + t) * 8;
      fast_vec<T, G>(p.w.p, k < p.N ? k : 0, held[2 * c]);
      fast_vec<T, G>(p.b.p, k < p.N ? k : 0, held[2 * c + 1]);
    }
  }
  for (uint32_t turn = 0; row < p.M; row += step, turn ^= 1u) {
    uint64_t v[NC][4], s2 = 0ull, q2 = 0ull;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      pairs_of<T>(w[c], v[c]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = add2(s2, v[c][i]);
    }
    if (row + step < p.M) fetch(row + step);
    float mean = rows::warp_sum(sum_of(s2)) * inv_mine, q;
    const uint64_t minus = both(-mean);
    if (G || all) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (!G || (c * width + t) * 8 < p.N)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t d = add2(v[c][i], minus);
            q2 = pipe::fma2(d, d, q2);
          }
    } else {  // the same without the values that the row does not have
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int n = p.N - (c * width + t) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float d, e;
          pipe::unpack2(add2(v[c][i], minus), d, e);
          const uint64_t f = pipe::pack2(2 * i < n ? d : 0.0f, 2 * i + 1 < n ? e : 0.0f);
          q2 = pipe::fma2(f, f, q2);
        }
      }
    }
    q = sum_of(q2);
    q = rows::warp_sum(q);
    if constexpr (!WARP) {
      if (lane == 0) part[turn][warp] = make_float2(mean, q);
      __syncthreads();
      mean = 0.0f;
      for (int i = 0; i < warps; ++i) mean += part[turn][i].x * counts[i];
      mean *= inv;
      q = 0.0f;
      for (int i = 0; i < warps; ++i) {
        const float2 u = part[turn][i];
        const float d = u.x - mean;
        q += u.y + counts[i] * (d * d);
      }
    }
    const float rstd = 1.0f / sqrtf(q * inv + p.eps);
    if (t == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    uint8_t* y = p.y + row * p.ldy;
    const uint64_t m2 = both(-mean), r2 = both(rstd);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (c * width + t) * 8;
      uint64_t g[4], b[4], o[4];
      if constexpr (G) {
        if (k >= p.N) continue;
        if constexpr (HOLD) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[i] = held[2 * c][i];
            b[i] = held[2 * c + 1][i];
          }
        } else {
          fast_vec<T, G>(p.w.p, k, g);
          fast_vec<T, G>(p.b.p, k, b);
        }
      } else {
        load_vec2(p.w, k, p.N, 1.0f, g);
        load_vec2(p.b, k, p.N, 0.0f, b);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = pipe::fma2(pipe::mul2(add2(v[c][i], m2), r2), g[i], b[i]);
      if constexpr (G) fast_store<T>(y + int64_t(k) * T::kBytes, o);
      else store_pairs(y + int64_t(k) * es, p.N - k, o, p.y_dtype, p.y_wide != 0);
    }
  }
}

// A CTA a row of any length, in loops.
template <typename T>
__global__ void __launch_bounds__(512) long_layer_norm_kernel(const FwdArgs p) {
  constexpr int TPR = 512;
  __shared__ float part[2][TPR / 32];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const int64_t row = blockIdx.x;
  const uint8_t* x = p.x.base + row * p.x.ld;
  const int es = p.y_dtype == SWZ_F32 ? 4 : 2;
  const float inv = 1.0f / float(p.N);
  // turns of the CTA, rounded up so that a warp's lanes stay together
  const int64_t turns = (p.N + int64_t(TPR) * 8 - 1) / (int64_t(TPR) * 8);
  uint32_t w[T::kWords];
  float s[1] = {0.0f};
  for (int64_t c = 0; c < turns; ++c) {
    const int64_t k = (c * TPR + threadIdx.x) * 8;
    rows::load8<T>(x + k * T::kBytes, p.N - k, p.x, w);
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) u += T::value(w, i);
    s[0] += u;
  }
  rows::row_sums<TPR, 1>(s, part[0]);
  const float mean = s[0] * inv;
  s[0] = 0.0f;
  for (int64_t c = 0; c < turns; ++c) {
    const int64_t k = (c * TPR + threadIdx.x) * 8;
    rows::load8<T>(x + k * T::kBytes, p.N - k, p.x, w);
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = T::value(w, i) - mean;
      u += k + i < p.N ? d * d : 0.0f;
    }
    s[0] += u;
  }
  rows::row_sums<TPR, 1>(s, part[1]);
  const float rstd = 1.0f / sqrtf(s[0] * inv + p.eps);
  if (threadIdx.x == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  for (int64_t c = 0; c < turns; ++c) {
    const int64_t k = (c * TPR + threadIdx.x) * 8;
    rows::load8<T>(x + k * T::kBytes, p.N - k, p.x, w);
    float g[8], b[8], o[8];
    load_vec(p.w, k, p.N, 1.0f, g);
    load_vec(p.b, k, p.N, 0.0f, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (T::value(w, i) - mean) * rstd * g[i] + b[i];
    rows::store8(p.y + row * p.ldy + k * es, p.N - k, o, p.y_dtype, p.y_wide != 0);
  }
}

template <typename T, int NC, bool WARP, int G, int MOST>
static int start_kind(const FwdArgs& a, int num_sms, cudaStream_t s) {
  const int threads = WARP ? 256 : threads_of(a.N, NC);
  int resident = 0;
  const int rc = resident_ctas<layer_norm_kernel<T, NC, WARP, G, MOST>>(threads, &resident);
  if (rc != SWZ_OK) return rc;
  const int64_t rows = WARP ? (int64_t(a.M) + 7) / 8 : int64_t(a.M);
  const int64_t most = int64_t(num_sms) * resident;
  return launch(layer_norm_kernel<T, NC, WARP, G, MOST>, uint32_t(rows < most ? rows : most), uint32_t(threads), a, s);
}

template <typename T, int NC, bool WARP, int MOST>
static int start(const FwdArgs& a, int num_sms, cudaStream_t s) {
  const int g = kind_of<T>(a.w);
  if (g == 0 || g != kind_of<T>(a.b) || !a.x.wide || !a.y_wide || a.N % 8 != 0 ||
      a.y_dtype != code_of<T>())
    return start_kind<T, NC, WARP, 0, MOST>(a, num_sms, s);
  if constexpr (T::kBytes == 2)
    if (g == 2) return start_kind<T, NC, WARP, 2, MOST>(a, num_sms, s);
  return start_kind<T, NC, WARP, 1, MOST>(a, num_sms, s);
}

template <typename T>
static int dispatch(const FwdArgs& a, int num_sms, cudaStream_t s) {
  if (a.N <= 256) return start<T, 1, true, 256>(a, num_sms, s);
  if (a.N <= 512) return start<T, 2, true, 256>(a, num_sms, s);
  if (a.N <= 4096) return start<T, 2, false, 256>(a, num_sms, s);
  if (a.N <= 8192) return start<T, 2, false, 512>(a, num_sms, s);
  if (a.N <= 16384) return start<T, 4, false, 512>(a, num_sms, s);
  return launch(long_layer_norm_kernel<T>, uint32_t(a.M), 512, a, s);
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
  const RowsInMemory result = rows_at(y, y_dtype, ldy, M, N);
  if (!may_lie(result, y_dtype, rows_at(x, dtype, ldx, M, N), dtype) ||
      !apart(result, weight, N * size_of(w_dtype)) || !apart(result, bias, N * size_of(b_dtype)))
    return SWZ_EINVAL;
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
  if (dtype == SWZ_BF16) return dispatch<rows::Bf16>(a, dev.num_sms, s);
  if (dtype == SWZ_F16) return dispatch<rows::F16>(a, dev.num_sms, s);
  return dispatch<rows::F32>(a, dev.num_sms, s);
}
