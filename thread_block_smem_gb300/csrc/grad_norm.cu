// grad_norm.cu -- the norm of all gradients of a network together, and their
// clipping:
//     norm = sqrt(sum over the tensors of sum g^2)
//     out = g min(1, max_norm / (norm + eps))
//
// The tensors come as a list; a launch carries their pointers and sizes in its
// parameters (no copy to the device, nothing kept between calls, and a captured
// launch has its own).  All elements are cut into pieces, dealt out to the CTAs.
//
// Sums: a piece's squares are added in fp32 by each thread (64 of them, two sums of
// 32), a thread's pieces in two fp32 numbers, everything above in 64 bits, in an order
// that depends on the sizes alone.  Squares leave fp32's range long before the
// gradients do, so eight values at a time whose largest magnitude is not within
// 2^-40 .. 2^50 are squared after a multiplication by 2^80 or 2^-80 and kept apart.
//
// Bound: memory: every gradient is read for the norm, read again and written.  The
// second pass takes the pieces in the opposite order, so that what the first one read
// last is still in L2.
//
// Measured: 671 M bf16 into fp32 837 us (792 at the copy bandwidth, 594 with one read),
// the norm alone 207 (198); 33.6 M 65 (40); 1.2 M fp32 8.3 (1.5: two launches).  With a
// thread's pieces added in 64 bits, of which the SM does a few a clock, the norm took
// 284 us; pieces of two chunks a thread instead of eight 498; the second pass with eight
// instead of four 894.
#include <algorithm>
#include <vector>

#include "common.h"
#include "pipe.cuh"
#include "rows.cuh"

namespace swz {
namespace grad {

constexpr int kThreads = 256;
// chunks of eight values a thread and piece, of the pass that adds and of that which
// scales (and has to hold its results)
constexpr int kAddTurns = 8, kScaleTurns = 4;
constexpr int64_t piece_of(int turns) { return int64_t(kThreads) * turns * 8; }
constexpr int kMaxBlocks = 1216;                   // partial sums of one launch
constexpr int kFew = 32, kMany = 1000;             // tensors a launch carries

struct Tensor {
  const uint8_t* in;
  uint8_t* out;
  int64_t n;
  uint32_t first;  // its first piece
  uint8_t in_dtype, out_dtype, in_wide, out_wide;
};

template <int CAP>
struct Table {
  Tensor t[CAP];
  int count;
  uint32_t pieces;
  const double* parts;  // partial sums of all launches
  int part_count;
  double* mine;         // where this launch's go
  double max_norm, eps;
  float* norm;
};
static_assert(sizeof(Table<kMany>) <= 32764, "kernel parameters");

// the tensor that piece `i` belongs to; `was`: the one of the piece before
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& p, uint32_t i, int was) {
  if (p.t[was].first <= i && (was + 1 == p.count || i < p.t[was + 1].first)) return was;
  int lo = 0, hi = p.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.t[mid].first <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float sum_of(uint64_t v) {
  float a, b;
  pipe::unpack2(v, a, b);
  return a + b;
}

// Sums of squares, two at a time: as they are, and of what was scaled down or up.
struct Squares {
  uint64_t mid = 0ull, high = 0ull, low = 0ull;
};

template <typename T>
__device__ __forceinline__ void add_squares(const uint32_t* w, Squares& s) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < T::kWords; ++j) m = f8::max_packed<T>(m, w[j] & T::kAbs);
  if constexpr (T::kBytes == 2) m = max(m & 0xFFFFu, m >> 16);
  const uint32_t bits = T::max_bits(m);
  constexpr uint32_t kLow = (127 - 40) << 23, kHigh = (127 + 50) << 23;
  uint64_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pipe::pack2(T::value(w, 2 * i), T::value(w, 2 * i + 1));
  if (bits < kHigh && (bits >= kLow || m == 0)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s.mid = pipe::fma2(v[i], v[i], s.mid);
  } else {
    const bool up = bits < kLow;
    const uint64_t f = up ? pipe::pack2(0x1p80f, 0x1p80f) : pipe::pack2(0x1p-80f, 0x1p-80f);
    uint64_t q = up ? s.low : s.high;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x = pipe::mul2(v[i], f);
      q = pipe::fma2(x, x, q);
    }
    (up ? s.low : s.high) = q;
  }
}

// The chunks of a piece that this thread takes: whole ones at 16-byte addresses, or any.
template <typename T, int TURNS>
__device__ __forceinline__ void load_piece(const Tensor& t, int64_t at,
                                           uint32_t (&w)[TURNS][T::kWords]) {
  const uint8_t* p = t.in + (at + int64_t(threadIdx.x) * 8) * T::kBytes;
  if (t.in_wide && at + piece_of(TURNS) <= t.n) {
#pragma unroll
    for (int j = 0; j < TURNS; ++j)
#pragma unroll
      for (int i = 0; i < T::kWords / 4; ++i)
        rows::ld16(p + j * (kThreads * 8 * T::kBytes) + 16 * i, w[j] + 4 * i);
    return;
  }
  rows::Span m{t.in, t.in + t.n * T::kBytes, 0, t.in_wide};
#pragma unroll
  for (int j = 0; j < TURNS; ++j) {
    const int64_t k = at + (int64_t(j) * kThreads + threadIdx.x) * 8;
    rows::load8<T>(t.in + k * T::kBytes, t.n - k, m, w[j]);
  }
}

// The pieces' sums of squares in a thread: two fp32 numbers, the second what the first's
// additions rounded off (64-bit additions, a few a clock and SM, took as long as reading
// a piece), and in 64 bits what was scaled.
struct Total {
  float sum = 0.0f, rest = 0.0f;
  double scaled = 0.0;
};

template <typename T>
__device__ __forceinline__ void piece_squares(const Tensor& t, int64_t at, Total& s) {
  uint32_t w[kAddTurns][T::kWords];
  load_piece<T, kAddTurns>(t, at, w);
  Squares q;
#pragma unroll
  for (int j = 0; j < kAddTurns; ++j) add_squares<T>(w[j], q);
  const float x = sum_of(q.mid), sum = s.sum + x, part = sum - s.sum;
  s.rest += (s.sum - (sum - part)) + (x - part);
  s.sum = sum;
  const float low = sum_of(q.low), high = sum_of(q.high);
  if (low != 0.0f) s.scaled += double(low) * 0x1p-160;
  if (!(high == 0.0f)) s.scaled += double(high) * 0x1p160;
}

// Sum over the CTA, the same bits in every thread.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) v += part[i];
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<CAP> p) {
  __shared__ double part[kThreads / 32];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  Total total;
  int which = 0;
  for (uint32_t i = blockIdx.x; i < p.pieces; i += gridDim.x) {
    which = tensor_of(p, i, which);
    const Tensor& t = p.t[which];
    const int64_t at = int64_t(i - t.first) * piece_of(kAddTurns);
    if (t.in_dtype == SWZ_BF16) piece_squares<rows::Bf16>(t, at, total);
    else if (t.in_dtype == SWZ_F16) piece_squares<rows::F16>(t, at, total);
    else piece_squares<rows::F32>(t, at, total);
  }
  const double s =
      block_sum(double(total.sum) + double(total.rest) + total.scaled, part);
  if (threadIdx.x == 0) p.mine[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ void scale_piece(const Tensor& t, int64_t at, float f) {
  uint32_t w[kScaleTurns][T::kWords];
  load_piece<T, kScaleTurns>(t, at, w);
  const uint64_t f2 = pipe::pack2(f, f);
  const int es = t.out_dtype == SWZ_F32 ? 4 : 2;
  uint8_t* p = t.out + (at + int64_t(threadIdx.x) * 8) * es;
  const bool whole = t.out_wide && at + piece_of(kScaleTurns) <= t.n;
#pragma unroll
  for (int j = 0; j < kScaleTurns; ++j) {
    uint64_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pipe::mul2(pipe::pack2(T::value(w[j], 2 * i), T::value(w[j], 2 * i + 1)), f2);
    uint8_t* const to = p + int64_t(j) * (kThreads * 8) * es;
    if (whole && t.out_dtype == SWZ_F32) {
      reinterpret_cast<ulonglong2*>(to)[0] = make_ulonglong2(v[0], v[1]);
      reinterpret_cast<ulonglong2*>(to)[1] = make_ulonglong2(v[2], v[3]);
      continue;
    }
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) pipe::unpack2(v[i], o[2 * i], o[2 * i + 1]);
    if (whole) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = rows::pack16(o[2 * i], o[2 * i + 1], t.out_dtype);
      *reinterpret_cast<uint4*>(to) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      rows::store8(to, t.n - (at + (int64_t(j) * kThreads + threadIdx.x) * 8), o, t.out_dtype,
                   t.out_wide != 0);
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<CAP> p) {
  __shared__ double part[kThreads / 32];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  double s = 0.0;
  for (int i = int(threadIdx.x); i < p.part_count; i += kThreads) s += p.parts[i];
  s = block_sum(s, part);
  __shared__ float factor;
  if (threadIdx.x == 0) {  // 64-bit roots and divisions are slow here: one thread's
    const double norm = sqrt(s);
    if (p.norm && blockIdx.x == 0) *p.norm = float(norm);
    // of the norm in 64 bits: one that fp32 cannot hold still clips.  A NaN stays one:
    // the comparison is false.
    const double den = norm + p.eps, quotient = den == 0.0 ? 1.0 : p.max_norm / den;
    factor = quotient > 1.0 ? 1.0f : float(quotient);
  }
  __syncthreads();
  const float f = factor;
  int which = p.count - 1;
  for (uint32_t j = blockIdx.x; j < p.pieces; j += gridDim.x) {
    const uint32_t i = p.pieces - 1 - j;
    which = tensor_of(p, i, which);
    const Tensor& t = p.t[which];
    if (f == 1.0f && t.in == t.out) continue;  // in place, nothing changes
    const int64_t at = int64_t(i - t.first) * piece_of(kScaleTurns);
    if (t.in_dtype == SWZ_BF16) scale_piece<rows::Bf16>(t, at, f);
    else if (t.in_dtype == SWZ_F16) scale_piece<rows::F16>(t, at, f);
    else scale_piece<rows::F32>(t, at, f);
  }
}

static int64_t size_of(int dtype) { return dtype == SWZ_F32 ? 4 : 2; }
static bool float_type(int d) { return d == SWZ_F16 || d == SWZ_BF16 || d == SWZ_F32; }

template <typename Kernel, typename Args>
static int launch(Kernel k, uint32_t grid, const Args& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, k, a));
  return SWZ_OK;
}

// No result may lie over another tensor's values, or over its own in another form.
static bool apart(const swz_grad* g, int count) {
  struct Range {
    uintptr_t from, to;
    bool written;
  };
  std::vector<Range> r;
  r.reserve(size_t(count) * 2);
  for (int i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uintptr_t in = reinterpret_cast<uintptr_t>(g[i].in);
    const uintptr_t out = reinterpret_cast<uintptr_t>(g[i].out);
    r.push_back({out, out + uintptr_t(g[i].n * size_of(g[i].out_dtype)), true});
    if (in != out || g[i].dtype != g[i].out_dtype)
      r.push_back({in, in + uintptr_t(g[i].n * size_of(g[i].dtype)), false});
  }
  auto before = [](const Range& a, const Range& b) { return a.from < b.from; };
  if (!std::is_sorted(r.begin(), r.end(), before)) std::sort(r.begin(), r.end(), before);
  uintptr_t read = 0, written = 0;  // ends of what came before
  for (const Range& x : r) {
    if (x.from < written || (x.written && x.from < read)) return false;
    uintptr_t& end = x.written ? written : read;
    end = std::max(end, x.to);
  }
  return true;
}

template <int CAP>
static void fill(Table<CAP>* p, const swz_grad* g, int from, int to, bool clip, int turns) {
  uint64_t pieces = 0;
  p->count = 0;
  for (int i = from; i < to; ++i) {
    if (g[i].n == 0) continue;
    Tensor& t = p->t[p->count++];
    t.in = static_cast<const uint8_t*>(g[i].in);
    t.out = clip ? static_cast<uint8_t*>(g[i].out) : nullptr;
    t.n = g[i].n;
    t.first = uint32_t(pieces);
    t.in_dtype = uint8_t(g[i].dtype);
    t.out_dtype = uint8_t(g[i].out_dtype);
    t.in_wide = aligned16(t.in);
    t.out_wide = aligned16(t.out);
    pieces += uint64_t((g[i].n + piece_of(turns) - 1) / piece_of(turns));
  }
  p->pieces = uint32_t(pieces);
}

template <int CAP>
static int run(const swz_grad* g, int count, bool clip, double max_norm, double eps, float* norm,
               double* parts, int num_sms, cudaStream_t s) {
  Table<CAP> p{};
  p.parts = parts;
  p.max_norm = max_norm;
  p.eps = eps;
  int blocks = num_sms * 8;
  if (blocks > kMaxBlocks) blocks = kMaxBlocks;
  for (int from = 0; from < count; from += CAP) {
    fill(&p, g, from, std::min(count, from + CAP), clip, kAddTurns);
    if (p.count == 0) continue;
    p.mine = parts + p.part_count;
    const uint32_t grid = std::min(p.pieces, uint32_t(blocks));
    const int rc = launch(squares_kernel<CAP>, grid, p, s);
    if (rc != SWZ_OK) return rc;
    p.part_count += int(grid);
  }
  // the norm alone, or that of no elements, is one CTA's work
  p.norm = norm;
  for (int from = 0; clip && from < count; from += CAP) {
    fill(&p, g, from, std::min(count, from + CAP), clip, kScaleTurns);
    if (p.count == 0) continue;
    const int rc = launch(scale_kernel<CAP>, std::min(p.pieces, uint32_t(blocks)), p, s);
    if (rc != SWZ_OK) return rc;
    p.norm = nullptr;
  }
  if (!p.norm) return SWZ_OK;
  p.count = 0;
  p.pieces = 0;
  return launch(scale_kernel<CAP>, 1, p, s);
}

static int check_and_run(const swz_grad* g, int count, bool clip, double max_norm, double eps,
                         float* norm, void* d_workspace, uint64_t workspace_bytes, void* stream) {
  if (count < 0 || (count > 0 && !g) || !norm || !aligned4(norm)) return SWZ_EINVAL;
  if (clip && (!(max_norm >= 0.0) || !(eps >= 0.0))) return SWZ_EINVAL;
  uint64_t pieces = 0;
  for (int i = 0; i < count; ++i) {
    if (g[i].n < 0 || g[i].n > (int64_t(1) << 44) || !float_type(g[i].dtype)) return SWZ_EINVAL;
    if (clip && !float_type(g[i].out_dtype)) return SWZ_EINVAL;
    if (g[i].n == 0) continue;
    if (!g[i].in || reinterpret_cast<uintptr_t>(g[i].in) % uintptr_t(size_of(g[i].dtype)))
      return SWZ_EINVAL;
    if (clip && (!g[i].out ||
                 reinterpret_cast<uintptr_t>(g[i].out) % uintptr_t(size_of(g[i].out_dtype))))
      return SWZ_EINVAL;
    pieces += uint64_t((g[i].n + piece_of(kScaleTurns) - 1) / piece_of(kScaleTurns));
    if (pieces > uint64_t(INT32_MAX)) return SWZ_EINVAL;
  }
  try {
    if (clip && !apart(g, count)) return SWZ_EINVAL;
  } catch (...) {  // no memory for the list of ranges
    return cuda_fail(cudaErrorMemoryAllocation);
  }
  uint64_t need = 0;
  const int rs = swz_grad_norm_workspace_size(count, &need);
  if (rs != SWZ_OK) return rs;
  if (need && (!d_workspace || !aligned16(d_workspace) || workspace_bytes < need))
    return SWZ_EINVAL;
  DeviceInfo dev{};
  const int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* parts = static_cast<double*>(d_workspace);
  return count <= kFew
             ? run<kFew>(g, count, clip, max_norm, eps, norm, parts, dev.num_sms, s)
             : run<kMany>(g, count, clip, max_norm, eps, norm, parts, dev.num_sms, s);
}

}  // namespace grad
}  // namespace swz

using namespace swz;
using namespace swz::grad;

extern "C" int swz_grad_norm_workspace_size(int count, uint64_t* h_bytes) {
  if (!h_bytes || count < 0) return SWZ_EINVAL;
  *h_bytes = (uint64_t(count) + kMany - 1) / kMany * kMaxBlocks * sizeof(double);
  return SWZ_OK;
}

extern "C" int swz_grad_norm(const swz_grad* grads, int count, float* norm, void* d_workspace,
                             uint64_t workspace_bytes, void* stream) {
  return check_and_run(grads, count, false, 0.0, 0.0, norm, d_workspace, workspace_bytes, stream);
}

extern "C" int swz_clip_grad_norm(const swz_grad* grads, int count, double max_norm, double eps,
                                  float* norm, void* d_workspace, uint64_t workspace_bytes,
                                  void* stream) {
  return check_and_run(grads, count, true, max_norm, eps, norm, d_workspace, workspace_bytes,
                       stream);
}
