// newton_schulz_small.cu -- swz_newton_schulz for matrices with a short side
// of up to 128 and a long one of up to 2048: all steps in one kernel.
//
// Bound: latency.  In kernels of their own three products a step cost 3 to 6 us a
// launch, 54 to 85 us for five steps, whatever the size.
// Here a cluster of 1 to 8 CTAs holds a matrix: each CTA has the d short rows
// of X and up to 256 of its long columns in shared memory and TMEM, and
//   P = X X^T     is summed over the cluster (each rank adds its share of the
//                 rows through distributed shared memory and hands A to all),
//   A A           is computed by every CTA for itself,
//   a X + B X     accumulates in TMEM onto a X, which never leaves fp32.
// X is kept as the operands of both products at once: 128 rows of 64 fp16
// columns, 128-byte swizzle, read K-major for P and N-major for B X.
//
// Precision: X and B are held as two fp16 numbers each (22 bits), the third
// cross product left out; A as one.  The tensor core is idle most of the time
// here, and matrices this small average over few roundings: one fp16 each was
// 0.17 % off on 64 x 64, this is 0.06 %.
//
// Measured, five steps, bf16: 64 x 64 25 us against 54 in kernels of their own, 128 x
// 128 35 against 56, 128 x 512 51 against 64, 128 x 2048 74 against 85.  From one
// step and five: 10, 15, 16 and 26 us of these are there whatever the steps --
// launch, G (value by value: its rows start anywhere), norm, first X, result -- and
// a step takes 3.1, 4.0, 7.0 and 9.6 us.  A CTA of 128 columns alone takes 4.0 for it;
// in a cluster its sum adds 2 to 3.5: two barriers and the remote reads between
// them.  fp32 G: 24, 31, 48 (100 x 333) and 69 us (2048 x 128); tall bf16 ones take up
// to 13 us more than wide ones.
#include <math.h>

#include <mutex>
#include <type_traits>

#include "common.h"
#include "f8.cuh"
#include "newton_schulz.cuh"
#include "pipe.cuh"

namespace swz {
namespace ns {

constexpr int kSmallWarps = 8;
constexpr int kSmallCols = 256;  // of a CTA
constexpr uint32_t kAtom = 128 * 128;  // bytes of 128 rows x 64 fp16 columns
// X high and low; A; B high and low, where the partial sums of P also go
constexpr uint32_t kOffXl = kSmallCols / 64 * kAtom, kOffA = 2 * kOffXl, kOffB = kOffA + 2 * kAtom;
constexpr uint32_t kSmallSmem = 1024 + kOffB + 4 * kAtom + 256;
static_assert(kSmallSmem <= 227 * 1024, "shared memory");
// TMEM: X (256 columns), P and A A (128)
constexpr uint32_t kTmemP = kSmallCols, kSmallTmem = 512;

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// byte offset of eight columns from `col` (a multiple of 8) of row `row`
__device__ __forceinline__ uint32_t at8(uint32_t row, uint32_t col) {
  return (col / 64) * kAtom + row * 128 + (((col % 64) / 8) ^ (row & 7u)) * 16;
}

// y[0 .. 31] as two fp16 numbers each: columns col .. of row `row` of the
// matrices at `high` and `low`
__device__ __forceinline__ void put_split(uint32_t high, uint32_t low, uint32_t row, uint32_t col,
                                          const float (&y)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = y[8 * c + 2 * j], b = y[8 * c + 2 * j + 1];
      h[j] = half2_bits(a, b);
      const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      l[j] = half2_bits(a - back.x, b - back.y);
    }
    const uint32_t o = at8(row, col + 8 * c);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(high + o), "r"(h[0]), "r"(h[1]),
                 "r"(h[2]), "r"(h[3])
                 : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(low + o), "r"(l[0]), "r"(l[1]),
                 "r"(l[2]), "r"(l[3])
                 : "memory");
  }
}

__global__ void __launch_bounds__(kSmallWarps * 32, 1)
    ns_small_kernel(const __grid_constant__ SmallParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sX = ptx::smem_u32(smem), sXl = sX + kOffXl, sA = sX + kOffA, sB = sX + kOffB;
  const uint32_t sBl = sB + 2 * kAtom;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffB + 4 * kAtom);
  double* part = reinterpret_cast<double*>(bars + 2);       // [3] this CTA's sums of squares
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(part + 3);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  Scale* sc_slot = reinterpret_cast<Scale*>(abort_flag + 1);
  double(*warp_part)[3] = reinterpret_cast<double(*)[3]>(smem + kOffB);  // [warp]
  const uint32_t bar = ptx::smem_u32(bars), drain_bar = bar + 8;
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0);
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t S = p.ranks;
  const uint32_t rank = S > 1 ? ptx::cluster_ctarank() : 0u;
  const uint32_t b = blockIdx.x / S;
  if (threadIdx.x == 0) {
    ptx::mbar_init(bar, 1);
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc<1>(ptx::smem_u32(tmem_slot), kSmallTmem);
    ptx::tmem_relinquish<1>();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (S > 1) ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pipe::Ctl ctl;
  ctl.status = p.status;
  ctl.abort_flag = abort_flag;
  ctl.peer_abort = 0;
  ctl.timeout_ns = p.timeout_ns;
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();

  // This thread: short row `row`, half `half` of the CTA's columns (in chunks
  // of 32); of P, A and B the columns 64 half ..
  const uint32_t q = warp & 3u, half = warp >> 2;
  const uint32_t row = q * 32 + lane;
  const uint32_t lane_addr = (q * 32u) << 16;
  const int64_t long0 = int64_t(rank) * p.cols;  // first long index of this CTA
  const int es = p.g_dtype == SWZ_F32 ? 4 : 2, ys = p.y_dtype == SWZ_F32 ? 4 : 2;
  const uint8_t* g = p.g + (b * p.batch_g) * es;
  const uint32_t chunks = p.cols / 32;  // of this CTA, dealt out to the two halves
  // 32 elements of G from long index long0 + 32 c, this thread's short row;
  // a warp's loads run along G's rows
  auto load_g = [&](uint32_t c, float (&v)[32]) {
    const int64_t l0 = long0 + c * 32;
    if (p.wide) {
      const bool in = l0 + lane < p.len;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        v[j] = in && int(q * 32) + j < p.d
                   ? load_any(g, int64_t(q * 32 + j) * p.ld_g + l0 + lane, p.g_dtype)
                   : 0.f;
      pipe::transpose32(v, lane);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        v[j] = int(row) < p.d && l0 + j < p.len
                   ? load_any(g, (l0 + j) * p.ld_g + row, p.g_dtype)
                   : 0.f;
    }
  };

  // ---- G to TMEM as it is, and its norm, over the cluster ----------------------------
  {
    float s0 = 0.f, s1 = 0.f, s2 = 0.f;
    for (uint32_t c = half; c < chunks; c += 2) {
      float v[32];
      load_g(c, v);
      uint32_t d[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float lo = v[j] * 0x1p-80f, hi = v[j] * 0x1p80f;
        s0 = fmaf(v[j], v[j], s0);
        s1 = fmaf(lo, lo, s1);
        s2 = fmaf(hi, hi, s2);
        d[j] = __float_as_uint(v[j]);
      }
      __syncwarp();
      tmem_st32(tmem + lane_addr + c * 32, d);
    }
    tmem_st_wait();
    double d[3] = {s0, s1, s2};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
      for (int o = 16; o > 0; o /= 2) d[k] += __shfl_xor_sync(0xFFFFFFFFu, d[k], o);
      if (lane == 0) warp_part[warp][k] = d[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
      double v = 0.0;
      for (int w = 0; w < kSmallWarps; ++w) v += warp_part[w][threadIdx.x];
      part[threadIdx.x] = v;
    }
    __syncthreads();
    if (S > 1) ptx::cluster_sync();
    if (warp == 0) {
      // lane r has rank r's sums; added in rank order
      double v[3] = {0.0, 0.0, 0.0}, sum[3] = {0.0, 0.0, 0.0};
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (lane < S)
          asm volatile("ld.shared::cluster.f64 %0, [%1];"
                       : "=d"(v[k])
                       : "r"(ptx::map_to_rank(ptx::smem_u32(part + k), lane))
                       : "memory");
#pragma unroll
      for (int k = 0; k < 3; ++k)
        for (uint32_t r = 0; r < S; ++r) sum[k] += __shfl_sync(0xFFFFFFFFu, v[k], r);
      if (lane == 0) *sc_slot = make_scale(sum, double(p.d) * double(p.len), p.eps, p.headroom);
    }
    __syncthreads();
  }
  const Scale sc = *sc_slot;

  uint32_t phase = 0;  // of `bar`
  // waits for the MMAs issued since the last wait
  auto done = [&]() {
    pipe::wait(bar, phase, ctl);
    phase ^= 1u;
    __syncwarp();
    ptx::tc_fence_after();
  };
  // what this thread wrote -- shared memory and TMEM -- before the next MMAs
  auto ready = [&]() {
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
  };

  // ---- the first X: fp16 pairs, and a X in TMEM ------------------------------------
  for (uint32_t c = half; c < chunks; c += 2) {
    float v[32];
    uint32_t d[32];
    ptx::tmem_ld_32x32b_x32(tmem + lane_addr + c * 32, d);
    pipe::tmem_ld_wait32(d);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = __uint_as_float(d[j]) * sc.p1 * sc.p2;
      d[j] = __float_as_uint(v[j] * p.ad[0]);
    }
    put_split(sX, sXl, row, c * 32, v);
    tmem_st32(tmem + lane_addr + c * 32, d);
  }
  tmem_st_wait();
  ready();

  const uint64_t dXk = pipe::sdesc128(sX, 16, 1024), dXlk = pipe::sdesc128(sXl, 16, 1024);
  const uint64_t dXn = pipe::sdesc128(sX, kAtom, 1024), dXln = pipe::sdesc128(sXl, kAtom, 1024);
  const uint64_t dA = pipe::sdesc128(sA, 16, 1024);
  const uint64_t dB = pipe::sdesc128(sB, 16, 1024), dBl = pipe::sdesc128(sBl, 16, 1024);
  const uint32_t id_p = pipe::idesc(0, 0, false, false, 128, 128);
  const uint32_t id_x = pipe::idesc(0, 0, false, true, 128, int(p.cols));
  // slice kk of 16 elements of K, in 16-byte units: K-major 32 bytes into atom
  // kk / 4; N-major 16 rows of 128 bytes down
  auto km = [](uint32_t kk) { return uint64_t((kk / 4) * (kAtom >> 4) + (kk % 4) * 2); };
  bool skip = (p.debug_flags & SWZ_DEBUG_SKIP_FIRST_LOAD) != 0;

  for (int i = 0; i < p.steps; ++i) {
    const float inv = i == 0 ? sc.f : sc.down;  // X over what the operands hold, but for 2^ex
    // ---- P = X X^T ----
    if (warp == 0 && pipe::elect_one() && !skip) {
      for (uint32_t kk = 0; kk < p.cols / 16; ++kk) {
        ptx::mma<1, 0>(tmem + kTmemP, dXk + km(kk), dXk + km(kk), id_p, kk != 0);
        ptx::mma<1, 0>(tmem + kTmemP, dXk + km(kk), dXlk + km(kk), id_p, 1u);
        ptx::mma<1, 0>(tmem + kTmemP, dXlk + km(kk), dXk + km(kk), id_p, 1u);
      }
      ptx::mma_commit(bar);
    }
    __syncwarp();
    skip = false;
    done();
    const float fa = p.fa[i] * inv * inv;
    if (S == 1) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(tmem + lane_addr + kTmemP + half * 64 + c * 32, r);
        pipe::tmem_ld_wait32(r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = half2_bits(__uint_as_float(r[8 * k + 2 * j]) * fa,
                              __uint_as_float(r[8 * k + 2 * j + 1]) * fa);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           sA + at8(row, half * 64 + c * 32 + k * 8)),
                       "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                       : "memory");
        }
      }
      ready();
    } else {
      // partial sums to shared memory: 16-byte piece c of a row at c ^ (row mod 32)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(tmem + lane_addr + kTmemP + half * 64 + c * 32, r);
        pipe::tmem_ld_wait32(r);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t piece = (half * 16 + c * 8 + k) ^ (row & 31u);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sB + row * 512 + piece * 16),
                       "r"(r[4 * k]), "r"(r[4 * k + 1]), "r"(r[4 * k + 2]), "r"(r[4 * k + 3])
                       : "memory");
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      ptx::cluster_sync();
      ptx::tc_fence_after();
      // this rank's share of the rows: 16 / S rows a warp, four columns a lane,
      // so that 16 remote reads are in flight whatever S is; added in rank
      // order, and the sum as fp16 to every CTA's A
      auto reduce = [&](auto ranks) {
        constexpr uint32_t R = decltype(ranks)::value, RW = 16 / R;
        float v[RW][R][4];
#pragma unroll
        for (uint32_t k = 0; k < RW; ++k) {
          const uint32_t r = rank * (128 / R) + warp * RW + k;
          const uint32_t from = sB + r * 512 + ((lane ^ (r & 31u)) << 4);
#pragma unroll
          for (uint32_t j = 0; j < R; ++j)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[k][j][0]), "=f"(v[k][j][1]), "=f"(v[k][j][2]), "=f"(v[k][j][3])
                         : "r"(ptx::map_to_rank(from, j))
                         : "memory");
        }
#pragma unroll
        for (uint32_t k = 0; k < RW; ++k) {
          float s[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[e] = v[k][0][e];
#pragma unroll
            for (uint32_t j = 1; j < R; ++j) s[e] += v[k][j][e];
          }
          const uint32_t h0 = half2_bits(s[0] * fa, s[1] * fa);
          const uint32_t h1 = half2_bits(s[2] * fa, s[3] * fa);
          const uint32_t r = rank * (128 / R) + warp * RW + k;
          const uint32_t to = sA + at8(r, lane / 2 * 8) + (lane % 2) * 8;
#pragma unroll
          for (uint32_t j = 0; j < R; ++j)
            asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(
                             ptx::map_to_rank(to, j)),
                         "r"(h0), "r"(h1)
                         : "memory");
        }
      };
      if (S == 2) reduce(std::integral_constant<uint32_t, 2>{});
      else if (S == 4) reduce(std::integral_constant<uint32_t, 4>{});
      else reduce(std::integral_constant<uint32_t, 8>{});
      fence_proxy_async_all();
      __syncwarp();
      ptx::cluster_sync();
      fence_proxy_async_all();
      ready();
    }

    // ---- A A, and B = b A + c A A as fp16 pairs ----
    if (warp == 0 && pipe::elect_one()) {
#pragma unroll
      for (uint32_t kk = 0; kk < 8; ++kk)
        ptx::mma<1, 0>(tmem + kTmemP, dA + km(kk), dA + km(kk), id_p, kk != 0);
      ptx::mma_commit(bar);
    }
    __syncwarp();
    done();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t r[32];
      ptx::tmem_ld_32x32b_x32(tmem + lane_addr + kTmemP + half * 64 + c * 32, r);
      float y[32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                     : "r"(sA + at8(row, half * 64 + c * 32 + k * 8))
                     : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
          y[8 * k + 2 * j] = p.ub[i] * z.x;
          y[8 * k + 2 * j + 1] = p.ub[i] * z.y;
        }
      }
      pipe::tmem_ld_wait32(r);
#pragma unroll
      for (int j = 0; j < 32; ++j) y[j] = fmaf(p.fb[i], __uint_as_float(r[j]), y[j]);
      put_split(sB, sBl, row, half * 64 + c * 32, y);
    }
    ready();

    // ---- X = a X + B X, onto a X ----
    if (warp == 0 && pipe::elect_one()) {
#pragma unroll
      for (uint32_t kk = 0; kk < 8; ++kk) {
        ptx::mma<1, 0>(tmem, dB + km(kk), dXn + 128 * kk, id_x, 1u);
        ptx::mma<1, 0>(tmem, dB + km(kk), dXln + 128 * kk, id_x, 1u);
        ptx::mma<1, 0>(tmem, dBl + km(kk), dXn + 128 * kk, id_x, 1u);
      }
      ptx::mma_commit(bar);
    }
    __syncwarp();
    done();
    const float k1 = p.k1[i] * inv;
    if (i + 1 < p.steps) {
      const float kx = k1 * p.sx[i + 1] * sc.up;
      for (uint32_t c = half; c < chunks; c += 2) {
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(tmem + lane_addr + c * 32, r);
        pipe::tmem_ld_wait32(r);
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          y[j] = __uint_as_float(r[j]) * kx;
          r[j] = __float_as_uint(y[j] * p.ad[i + 1]);
        }
        put_split(sX, sXl, row, c * 32, y);
        tmem_st32(tmem + lane_addr + c * 32, r);
      }
      tmem_st_wait();
      ready();
    } else {
      uint8_t* y = p.y + (b * p.batch_y) * ys;
      for (uint32_t c = half; c < chunks; c += 2) {
        uint32_t r[32];
        __syncwarp();
        ptx::tmem_ld_32x32b_x32(tmem + lane_addr + c * 32, r);
        pipe::tmem_ld_wait32(r);
        const int64_t l0 = long0 + c * 32;
        if (p.wide) {
          // rows of Y run along the long side: a lane a column
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * k1;
          pipe::transpose32(v, lane);
          if (l0 + lane < p.len)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (int(q * 32) + j < p.d)
                store_any(y, int64_t(q * 32 + j) * p.ld_y + l0 + lane, v[j], p.y_dtype);
        } else if (int(row) < p.d) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (l0 + j < p.len)
              store_any(y, (l0 + j) * p.ld_y + row, __uint_as_float(r[j]) * k1, p.y_dtype);
        }
      }
    }
  }

  // ---- teardown: every MMA has completed, also after a wait that ran out ----
  if (*reinterpret_cast<volatile int*>(abort_flag)) {
    if (warp == 0 && pipe::elect_one()) ptx::mma_commit(drain_bar);
    __syncwarp();
    const uint64_t t0 = ptx::global_timer_ns();
    while (!pipe::try_wait(drain_bar, 0) && ptx::global_timer_ns() - t0 < p.timeout_ns) {
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (S > 1) ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc<1>(tmem, kSmallTmem);
}

// As few ranks as hold the long side, 128 columns a rank while that is enough:
// an exchange over more of them costs more than the columns.
static uint32_t ranks_of(int len) {
  uint32_t ranks = 1;
  while (ranks < 8 && int64_t(ranks) * 128 < len) ranks *= 2;
  return ranks;
}

static cudaLaunchConfig_t config(int batch, uint32_t ranks, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(batch) * ranks);
  cfg.blockDim = dim3(kSmallWarps * 32);
  cfg.dynamicSmemBytes = kSmallSmem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Waves of matrices that run at a time, by the ranks of one, against the
// products' launches, whose time grows with the matrices.  Measured (one kernel,
// launches; us, five steps): 64 x 64 25, 54; 128 x 128 35, 56; 600 of them 138, 233;
// 128 x 256 47, 61; 152 of them (two waves) 96, 122; 40 of 100 x 512 (two waves) 102,
// 96; 128 x 1024 54, 71; 14 of 128 x 1100 67, 105; 128 x 2048 74, 85; 64 of them 375, 250.
// The rule weighs five steps, the usual number: of a single one the launches
// take up to 12 us less from 128 columns on (128 x 128 18 to 19, 128 x 512 19 to 23, 128 x
// 2048 23 to 35).
int small_pays(int batch, int len, bool* pays) {
  static std::mutex mu;
  static int resident[64][4] = {};  // clusters of 1, 2, 4, 8 at a time
  int dev = 0;
  SWZ_CUDA_TRY(cudaGetDevice(&dev));
  const uint32_t ranks = ranks_of(len);
  const int at = ranks == 1 ? 0 : ranks == 2 ? 1 : ranks == 4 ? 2 : 3;
  int fit;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (resident[dev][at] == 0) {
      SWZ_CUDA_TRY(cudaFuncSetAttribute(ns_small_kernel,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem));
      cudaLaunchAttribute attr[2];
      const cudaLaunchConfig_t cfg = config(1, ranks, attr);
      SWZ_CUDA_TRY(cudaOccupancyMaxActiveClusters(&resident[dev][at], ns_small_kernel, &cfg));
      if (resident[dev][at] < 1) resident[dev][at] = 1;
    }
    fit = resident[dev][at];
  }
  const double waves = double((batch + fit - 1) / fit);
  const double wave[4] = {35.0, 47.0, 51.0, 44.0 + 0.016 * len};
  *pays = waves * wave[at] <= 57.0 + 0.0135 * len + batch * (0.12 + 0.0009 * len);
  return SWZ_OK;
}

// After small_pays, which prepares the kernel on the device.
int launch_small(SmallParams p, int batch, cudaStream_t stream) {
  p.ranks = ranks_of(p.len);
  p.cols = uint32_t((((int64_t(p.len) + p.ranks - 1) / p.ranks) + 63) / 64 * 64);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config(batch, p.ranks, attr);
  cfg.stream = stream;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, ns_small_kernel, p));
  return SWZ_OK;
}

}  // namespace ns
}  // namespace swz
