// gemm_int8_tokens.cu -- swz_gemm_int8 and swz_linear_int8 with one or two rows of A
// (a decoding step), the same exact sums by dp4a.
//
// Bound: reading B once, N * K bytes.  A CTA takes a range of B's rows, the same
// number for all within one, and a warp of it a slot of K (512 bytes at a time, 16 a
// lane) of every `groups`-th of these rows.  A lane's 16 bytes of each row of A stay
// in registers for all of them, so that the inner loop is one load, four dp4a for
// each row of A, and one sum over the warp (redux) for each.  Eight rows' loads are
// in flight a warp.  The partial sums of the slots are added in shared memory: whole
// numbers, in any order.
//   * The layer quantises x here where it is short: every CTA needs all of it, and a
//     few thousand values are read and rounded while its first loads of B are under
//     way; a kernel of its own takes 1.8 us (and is what a result over x takes: other
//     CTAs store theirs while one still reads x).
//   * Rates on this GPU, multiply-adds a clock and SM: dp4a 255, mma.sync on 8-bit
//     integers 252, on fp16 1020.  B at the memory's rate asks for 24 a row of A.
//
// Measured, in a stream of them, B from memory: one row of 4096 x 4096 5.4 us
// (3.1 TB/s; 6.2 with x quantised here), 10240 x 4096 10.1 (4.2), 8192 x 8192 13.2
// (5.1); of the ring of gemm_int8_rows.cu 5.9, 10.6 and 14.2.  Two rows take 5.9, 11.4
// and 14.6 and the ring 5.9, 10.6 and 14.2, and a quantiser of its own before it; four
// rows 7.5, 13.5 and 18.2.
#include <type_traits>

#include "common.h"
#include "int8.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace swz {
namespace i8 {

constexpr int kTokWarps = 16, kTokThreads = kTokWarps * 32;
constexpr int kTokBytes = 32 * 1024;  // of x in shared memory, at most
constexpr uint32_t kTokRows = 1024;        // rows of B a CTA and turn

struct TokParams {
  const uint8_t* A;  // bytes; NULL: x is quantised here
  int64_t lda;
  rows::Span x;
  const uint8_t* B;
  int64_t ldb;
  const float *sa, *sb;
  uint8_t* C;
  int64_t ldc;  // elements
  int c_dtype;
  int M, N, K;
  uint32_t slots, groups;  // of K and of rows, slots * groups = kTokWarps
};

// the bytes of 16 that lie below K, for those from k on
__device__ __forceinline__ uint4 keep_below(uint4 v, int k, int K) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = K - k - 4 * i;  // of this word
    w[i] = n >= 4 ? w[i] : n <= 0 ? 0u : w[i] & (0xFFFFFFFFu >> (32 - 8 * n));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// MT: rows of A (the ones beyond M are zero); X: the type of x, void for bytes.
template <int MT, typename X>
__global__ void __launch_bounds__(kTokThreads, 2) gemm_int8_tokens_kernel(const TokParams p) {
  constexpr bool FUSED = !std::is_same<X, void>::value;
  constexpr int kAhead = 8;  // rows of B whose loads are in flight
  extern __shared__ uint4 tok_smem[];  // FUSED: x as bytes, rows of `pitch`
  __shared__ int32_t part[MT][kTokRows];
  __shared__ float scale[MT];
  __shared__ uint32_t wmax[MT][kTokWarps];
  uint8_t* const xq = reinterpret_cast<uint8_t*>(tok_smem);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t slot = warp % p.slots, group = warp / p.slots;
  const int pitch = (p.K + 15) / 16 * 16;
  // (rows are unsigned: with N just below 2^31 the loops go to numbers beyond it)
  const uint32_t n0 = uint32_t(int64_t(p.N) * blockIdx.x / gridDim.x);
  const uint32_t n1 = uint32_t(int64_t(p.N) * (blockIdx.x + 1) / gridDim.x);
  const int k0 = int(slot) * 512 + int(lane) * 16, k_step = int(p.slots) * 512;
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();

  // Every load is made, of rows and pieces that are there: rows beyond the range are not
  // summed, and what is beyond K meets zeros.
  uint4 b[kAhead];
  const int cut = p.K % 16 ? p.K - p.K % 16 : -1;  // the piece that K cuts
  auto fetch = [&](uint32_t n, int k) {
    if (k >= p.K || k == cut) k = 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t row = n + i * p.groups;
      b[i] = *reinterpret_cast<const uint4*>(p.B + int64_t(row < n1 ? row : n1 - 1) * p.ldb + k);
    }
  };
  fetch(n0 + group, k0);
  for (uint32_t i = threadIdx.x; i < MT * kTokRows; i += kTokThreads) (&part[0][0])[i] = 0;

  if constexpr (FUSED) {
    // as quantize_int8.cu: the row's maximum, then the exact product rounded once
    const int chunks = (p.K + 7) / 8;
    uint32_t m[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      m[t] = 0;
      if (t < p.M)
        for (int c = int(threadIdx.x); c < chunks; c += kTokThreads) {
          uint32_t w[X::kWords];
          rows::load8<X>(p.x.base + t * p.x.ld + int64_t(c) * 8 * X::kBytes, p.K - c * 8, p.x, w);
          m[t] = max(m[t], chunk_max<X>(w));
        }
      m[t] = __reduce_max_sync(0xFFFFFFFFu, m[t]);
      if (lane == 0) wmax[t][warp] = m[t];
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      uint32_t top = wmax[t][0];
#pragma unroll
      for (int i = 1; i < kTokWarps; ++i) top = max(top, wmax[t][i]);
      float r, s;
      const bool bad = row_scale(X::max_bits(top), r, s);
      if (threadIdx.x == 0) scale[t] = s;
      for (int c = int(threadIdx.x); c < 2 * ((chunks + 1) / 2); c += kTokThreads) {
        uint32_t w[X::kWords];
        rows::load8<X>(p.x.base + t * p.x.ld + int64_t(c) * 8 * X::kBytes,
                       t < p.M ? p.K - c * 8 : 0, p.x, w);
        store_q<X, false>(xq + t * pitch + c * 8, 8, w, r, bad);
      }
    }
  }
  __syncthreads();

  // whole turns of kTokRows rows: the partial sums of a turn fit shared memory
  for (uint32_t turn = n0; turn < n1; turn += kTokRows) {
    const uint32_t end = n1 - turn < kTokRows ? n1 : turn + kTokRows;
    for (int k = k0; k - int(lane) * 16 < p.K; k += k_step) {
      uint4 a[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        a[t] = make_uint4(0u, 0u, 0u, 0u);
        if (k < p.K && t < p.M) {
          if constexpr (FUSED) a[t] = *reinterpret_cast<const uint4*>(xq + t * pitch + k);
          else a[t] = keep_below(load_bytes(p.A + int64_t(t) * p.lda, k, p.K, t + 1 == p.M), k, p.K);
        }
      }
      for (uint32_t n = turn + group; n < end; n += kAhead * p.groups) {
        if (!(turn == n0 && k == k0 && n == n0 + group)) fetch(n, k);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t row = n + i * p.groups;
          if (row >= end) break;
          if (k == cut)
            b[i] = load_bytes(p.B + int64_t(row) * p.ldb, k, p.K, row + 1 == uint32_t(p.N));
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            int32_t s = __dp4a(int(b[i].x), int(a[t].x), 0);
            s = __dp4a(int(b[i].y), int(a[t].y), s);
            s = __dp4a(int(b[i].z), int(a[t].z), s);
            s = __dp4a(int(b[i].w), int(a[t].w), s);
            s = __reduce_add_sync(0xFFFFFFFFu, s);
            if (lane == uint32_t(t)) atomicAdd(&part[t][row - turn], s);
          }
        }
      }
    }
    __syncthreads();
    const int es = p.c_dtype == SWZ_F32 ? 4 : 2;
    const int cols = int(end - turn);
    for (int i = int(threadIdx.x); i < p.M * cols; i += kTokThreads) {
      const int t = i / cols, n = i % cols;
      const float sa = FUSED ? scale[t] : p.sa[t];
      const int64_t col = int64_t(turn) + n;
      rows::store1(p.C + (int64_t(t) * p.ldc + col) * es, float(part[t][n]) * (sa * p.sb[col]),
                   p.c_dtype);
      part[t][n] = 0;
    }
    __syncthreads();
  }
}

template <int MT, typename X>
static int launch_tokens(const TokParams& p, int num_sms, cudaStream_t s) {
  const uint64_t ctas = uint64_t(num_sms) * 2;
  cudaLaunchConfig_t cfg = {};
  // a CTA for every SM's half, or for as many rows as its groups take at once
  const uint64_t useful = (uint64_t(p.N) + p.groups - 1) / p.groups;
  cfg.gridDim = dim3(uint32_t(useful < ctas ? useful : ctas));
  cfg.blockDim = dim3(kTokThreads);
  cfg.dynamicSmemBytes = std::is_same<X, void>::value ? 0 : size_t(MT) * ((p.K + 15) / 16 * 16);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, gemm_int8_tokens_kernel<MT, X>, p));
  return SWZ_OK;
}

template <typename X>
static int launch_rows_of(const TokParams& p, int num_sms, cudaStream_t s) {
  return p.M == 1 ? launch_tokens<1, X>(p, num_sms, s) : launch_tokens<2, X>(p, num_sms, s);
}

// x short enough to be quantised by every CTA
bool tokens_fused(int M, int K) { return int64_t(M) * K <= kTokBytes; }

int gemm_int8_tokens(const void* A, int64_t lda, const float* sa, const void* x, int x_dtype,
                     int64_t ldx, const void* B, int64_t ldb, const float* sb, void* C,
                     int64_t ldc, int c_dtype, int M, int N, int K, int num_sms,
                     cudaStream_t stream) {
  TokParams p{};
  p.A = static_cast<const uint8_t*>(A);
  p.lda = lda;
  p.B = static_cast<const uint8_t*>(B);
  p.ldb = ldb;
  p.sa = sa;
  p.sb = sb;
  p.C = static_cast<uint8_t*>(C);
  p.ldc = ldc;
  p.c_dtype = c_dtype;
  p.M = M;
  p.N = N;
  p.K = K;
  for (p.slots = 1; p.slots < uint32_t(kTokWarps) && int64_t(p.slots) * 512 < K;) p.slots *= 2;
  p.groups = kTokWarps / p.slots;
  if (A) return launch_rows_of<void>(p, num_sms, stream);
  p.x = rows::span_of(x, x_dtype, ldx, M, K);
  if (x_dtype == SWZ_BF16) return launch_rows_of<rows::Bf16>(p, num_sms, stream);
  if (x_dtype == SWZ_F16) return launch_rows_of<rows::F16>(p, num_sms, stream);
  return launch_rows_of<rows::F32>(p, num_sms, stream);
}

}  // namespace i8
}  // namespace swz
