// gemm_int8.cu -- C = A * B^T of 8-bit integers with a scale for each row of A
// (token) and of B (output channel):
//     C[m, n] = sa[m] sb[n] * sum over k of A[m, k] B[n, k]
// A (M x K) and B (N x K) K-major; the sum is exact, C fp32, bf16 or fp16.
//
// Mathematics: the tensor cores of sm_103a take no 8-bit integers (tcgen05's
// kind::i8 is refused for this target), but fp16 holds every one of them exactly
// and an fp32 accumulator holds any sum of 1024 of their products exactly (2^14
// each, 2^24 in all).  So both operands are widened to fp16 by one pass of their
// own, the products run at the 16-bit rate, and each 1024 of K is an accumulation
// of its own, which is read back from TMEM as whole numbers and added in int32.
// The scales are applied to the total: sa sb is rounded once, the total once
// where it is above 2^24, their product once, and C once.
//   * One CTA per SM, 10 warps: 0-7 the sums and the epilogue (warp w: TMEM lanes
//     32 (w mod 4) .., half w / 4 of the tile's columns), 8 TMA producer, 9 MMA
//     issue and TMEM allocation.
//   * CTA pair: 256 x 256 (each CTA 128 rows of A and of B), stages of 64 of K, two
//     accumulators in TMEM; a chunk's MMAs take 8192 cycles, its way out of TMEM
//     about a quarter of that, under the next one's.  The totals are 128 int32
//     registers a thread.
//   * One CTA: 128 x 128, stages of 128 of K; a cluster of 1, 2, 4 or 8 shares a
//     tile's K and adds the partial tiles through distributed shared memory.
//   * Tiles are dealt out by the framework's tile orders, w = cluster + i P.
//
// Measured, both passes: 8192^3, bf16 result, 593 to 618 us over boxes (1.8 PFLOP/s), of
// which the pass that widens (134 MB read, 268 MB written) about 50; 8192 x 4096 x 4096
// 175 us; 1000 rows of 4096 x 4096 41.  Widening whole rows a warp took 610 us where
// parts of 2048 took 618, but 183 and 45 of the other two.  Bound: the tensor cores (pipe 85 % busy at 8192 x 4096 x
// 4096).
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "common.h"
#include "int8.cuh"
#include "ops.h"
#include "pipe.cuh"
#include "rows.cuh"
#include "tile_order.cuh"

namespace swz {
namespace i8 {

constexpr int kMath = 8;
constexpr int kThreads = (kMath + 2) * 32;
constexpr int kChunk = 1024;  // products whose sum fp32 holds exactly

template <bool PAIR>
struct Cfg {
  static constexpr int CG = PAIR ? 2 : 1;
  static constexpr int BN = PAIR ? 256 : 128;  // columns of the tile
  static constexpr int BN_LOCAL = 128;         // rows of B this CTA loads
  static constexpr int ATOMS = PAIR ? 1 : 2;   // pieces of 64 of K a stage
  static constexpr int BK = 64 * ATOMS;
  static constexpr int ATOM = 128 * 128;  // bytes: 128 rows of 128
  static constexpr int A_BYTES = ATOMS * ATOM, B_BYTES = ATOMS * ATOM;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = PAIR ? 6 : 3;
  static constexpr int NBUF = 512 / BN;
  static constexpr int COLS = BN / 2;  // columns a summing warp holds
  static constexpr int KB_CHUNK = kChunk / BK;
  static constexpr int BARS = 2 * STAGES + 2 * NBUF + 1;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + kMath * COLS * 4 + BARS * 8 + 16;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(STAGES * STAGE_BYTES >= 128 * BN * 4 || PAIR, "a partial tile fits the ring");
};

struct Params {
  void* C;
  int64_t ldc;
  const float *sa, *sb;
  int M, N;
  int c_dtype;
  int order;
  uint32_t group, sched_m, sched_n, num_kb, idesc, split;
  uint32_t c_align;  // bytes that every row start of C is a multiple of (32, 16 or less)
  uint32_t debug_flags;
  unsigned int* status;
  uint64_t timeout_ns;
};

// ---- widening -------------------------------------------------------------------
constexpr int kPart = 2048;  // values of a row that a warp widens at a time
struct WidenArgs {
  const uint8_t* in[2];
  int64_t ld[2];  // bytes
  uint8_t* out[2];
  int64_t ldo;  // bytes
  int rows[2];
  int K;
};

// Two matrices (either may be empty) of bytes to fp16: a warp takes 2048 values of a row at
// a time, four pieces of 16 a lane under way together.
__global__ void __launch_bounds__(256) widen_kernel(const WidenArgs p) {
  constexpr int kAhead = kPart / 512;
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const int lane = int(threadIdx.x % 32);
  const int64_t last = int64_t(p.rows[0]) + p.rows[1];
  // the warp's row and part of it, and how far the next ones are
  const int parts = (p.K + kPart - 1) / kPart;
  const int64_t at = int64_t(blockIdx.x) * 8 + threadIdx.x / 32, far = int64_t(gridDim.x) * 8;
  const int64_t far_rows = far / parts;
  const int far_parts = int(far % parts);
  int64_t r = at / parts;
  int part = int(at % parts);
  for (; r < last; r += far_rows, part += far_parts) {
    if (part >= parts) {
      part -= parts;
      if (++r >= last) break;
    }
    const int which = r >= p.rows[0];
    const int64_t row = which ? r - p.rows[0] : r;
    const uint8_t* src = p.in[which] + row * p.ld[which];
    uint8_t* dst = p.out[which] + row * p.ldo;
    const int k0 = part * kPart + lane * 16;
    uint32_t b[kAhead][4];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j * 512;
#pragma unroll
      for (int e = 0; e < 4; ++e) b[j][e] = 0u;
      if (k + 16 <= p.K) rows::ld16_once(src + k, b[j]);
      else if (k < p.K) {
        const uint4 v = load_bytes(src + k, 0, p.K - k, true);
        b[j][0] = v.x;
        b[j][1] = v.y;
        b[j][2] = v.z;
        b[j][3] = v.w;
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j * 512;
      if (k >= p.K) continue;
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) widen4(b[j][e], o[2 * e], o[2 * e + 1]);
      uint4* to = reinterpret_cast<uint4*>(dst + int64_t(k) * 2);
      to[0] = make_uint4(o[0], o[1], o[2], o[3]);
      to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// ---- product --------------------------------------------------------------------
template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmB, const Params p) {
  using K_ = Cfg<PAIR>;
  constexpr int CG = K_::CG, STAGES = K_::STAGES, NBUF = K_::NBUF, COLS = K_::COLS, BN = K_::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sA = ptx::smem_u32(smem);
  const uint32_t sB = sA + STAGES * K_::A_BYTES;
  float* const scales = reinterpret_cast<float*>(smem + STAGES * K_::STAGE_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(scales + kMath * COLS);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * STAGES + NBUF + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * NBUF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + K_::BARS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0);  // known uniform
  const uint32_t lane = threadIdx.x % 32;
  // rank: of a pair, which 128 rows of the tile; of a split, which range of K
  const uint32_t crank = (PAIR || p.split > 1) ? ptx::cluster_ctarank() : 0u;
  const uint32_t rank = PAIR ? crank : 0u;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tmA);
    ptx::prefetch_tensormap(&tmB);
    for (uint32_t s = 0; s < uint32_t(STAGES); ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (uint32_t a = 0; a < uint32_t(NBUF); ++a) {
      ptx::mbar_init(tfull_bar(a), 1);
      ptx::mbar_init(tempty_bar(a), kMath * CG);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMath + 1) {
    ptx::tmem_alloc<CG>(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish<CG>();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  pipe::Ctl ctl;
  ctl.status = p.status;
  ctl.abort_flag = abort_flag;
  ctl.peer_abort = 0;
  if constexpr (PAIR) ctl.peer_abort = ptx::map_to_rank(ptx::smem_u32(abort_flag), rank ^ 1u);
  ctl.timeout_ns = p.timeout_ns;

  const uint32_t units = p.sched_m * p.sched_n;
  const uint32_t cl = PAIR ? 2u : p.split;
  const uint32_t w0 = blockIdx.x / cl, P = gridDim.x / cl;
  uint32_t kb0 = 0, kb1 = p.num_kb;
  if (!PAIR && p.split > 1) {
    kb0 = uint32_t(uint64_t(p.num_kb) * crank / p.split);
    kb1 = uint32_t(uint64_t(p.num_kb) * (crank + 1) / p.split);
  }
  // nothing above touches global memory
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  bool aborted = false;

  if (warp == kMath) {
    // ---------------- TMA producer ----------------
    uint32_t stage = 0, phase = 0;
    bool skip = (p.debug_flags & SWZ_DEBUG_SKIP_FIRST_LOAD) != 0;
    const uint64_t pol = ptx::l2_policy_evict_last();
    const uint32_t full0 = PAIR ? ptx::map_to_rank(full_bar(0), 0) : full_bar(0);
    for (uint32_t w = w0; w < units && !aborted; w += P) {
      const TileCoord t = tile_of(p.order, w, p.sched_m, p.sched_n, p.group);
      const int32_t m0 = int32_t((t.m * CG + rank) * 128);
      const int32_t n0 = int32_t(t.n * BN + rank * K_::BN_LOCAL);
      for (uint32_t kb = kb0; kb < kb1; ++kb) {
        const bool ok = pipe::wait(empty_bar(stage), phase ^ 1u, ctl);
        if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
        if (pipe::elect_one()) {
          if (leader) ptx::mbar_arrive_expect_tx(full_bar(stage), CG * K_::STAGE_BYTES);
          if (!skip) {
            const uint32_t a_dst = sA + stage * K_::A_BYTES, b_dst = sB + stage * K_::B_BYTES;
#pragma unroll
            for (int h = 0; h < K_::ATOMS; ++h) {
              const int32_t k0 = int32_t(kb * K_::BK) + h * 64;
              if constexpr (PAIR) {
                ptx::tma_load_3d_pair(a_dst + h * K_::ATOM, &tmA, full0 + 8u * stage, k0, m0, 0, pol);
                ptx::tma_load_3d_pair(b_dst + h * K_::ATOM, &tmB, full0 + 8u * stage, k0, n0, 0, pol);
              } else {
                ptx::tma_load_3d(a_dst + h * K_::ATOM, &tmA, full0 + 8u * stage, k0, m0, 0, pol);
                ptx::tma_load_3d(b_dst + h * K_::ATOM, &tmB, full0 + 8u * stage, k0, n0, 0, pol);
              }
            }
          }
        }
        __syncwarp();
        skip = false;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    // every stage released: no commit is in flight towards this CTA
    for (int i = 0; i < STAGES && !aborted; ++i) {
      const bool ok = pipe::wait(empty_bar(stage), phase ^ 1u, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) aborted = true;
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    }
    if (aborted) pipe::spin_ns(50000);  // copies already issued land
    __syncwarp();
  } else if (warp == kMath + 1) {
    // ---------------- MMA issuer (leader CTA; one elected lane issues) ----------------
    if (leader) {
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
      bool issued = false;
      const uint64_t adesc0 = pipe::sdesc128(sA, 16, 1024);
      const uint64_t bdesc0 = pipe::sdesc128(sB, 16, 1024);
      for (uint32_t w = w0; w < units && !aborted; w += P) {
        uint32_t in_chunk = 0;  // blocks of K in the present accumulation
        for (uint32_t kb = kb0; kb < kb1; ++kb) {
          bool ok = pipe::wait(full_bar(stage), phase, ctl);
          if (ok && in_chunk == 0) ok = pipe::wait(tempty_bar(buf), buf_phase ^ 1u, ctl);
          if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
          ptx::tc_fence_after();
          const uint64_t a = adesc0 + uint64_t(stage * uint32_t(K_::A_BYTES >> 4));
          const uint64_t b = bdesc0 + uint64_t(stage * uint32_t(K_::B_BYTES >> 4));
          const uint32_t d = tmem_base + buf * BN;
          const bool last = in_chunk + 1 == uint32_t(K_::KB_CHUNK) || kb + 1 == kb1;
          if (pipe::elect_one()) {
#pragma unroll
            for (uint32_t h = 0; h < uint32_t(K_::ATOMS); ++h)
#pragma unroll
              for (uint32_t kk = 0; kk < 4; ++kk)
                ptx::mma<CG, 0>(d, a + h * (K_::ATOM >> 4) + kk * 2,
                                b + h * (K_::ATOM >> 4) + kk * 2, p.idesc,
                                (in_chunk | h | kk) != 0);
            if constexpr (PAIR) {
              ptx::mma_commit_pair(empty_bar(stage), 0x3);
              if (last) ptx::mma_commit_pair(tfull_bar(buf), 0x3);
            } else {
              ptx::mma_commit(empty_bar(stage));
              if (last) ptx::mma_commit(tfull_bar(buf));
            }
          }
          __syncwarp();
          issued = true;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          ++in_chunk;
          if (last) {
            in_chunk = 0;
            if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
          }
        }
      }
      if (aborted && issued) {
        // drain: wait (bounded) until every MMA issued so far has completed
        if (pipe::elect_one()) {
          if constexpr (PAIR) ptx::mma_commit_pair(drain_bar, 0x1);
          else ptx::mma_commit(drain_bar);
        }
        const uint64_t t0 = ptx::global_timer_ns();
        while (!pipe::try_wait(drain_bar, 0) && ptx::global_timer_ns() - t0 < p.timeout_ns) {
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------- sums and epilogue ----------------
    const uint32_t q = warp & 3u, part = warp >> 2;  // rows 32 q .., columns COLS part ..
    uint32_t buf = 0, buf_phase = 0;
    const uint32_t tempty0 = PAIR ? ptx::map_to_rank(tempty_bar(0), 0) : tempty_bar(0);
    const uint32_t taddr0 = tmem_base + ((q * 32u) << 16) + part * COLS;
    float* const sb = scales + warp * COLS;  // this warp's scales of B
    int32_t acc[COLS];
    for (uint32_t w = w0; w < units && !aborted; w += P) {
      const TileCoord t = tile_of(p.order, w, p.sched_m, p.sched_n, p.group);
      const int64_t row = int64_t(t.m * CG + rank) * 128 + q * 32 + lane;
      const int64_t col0 = int64_t(t.n) * BN + part * COLS;
      const float sa = row < p.M ? p.sa[row] : 0.0f;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < COLS / 32; ++j) {
        const int64_t n = col0 + j * 32 + lane;
        sb[j * 32 + lane] = n < p.N ? p.sb[n] : 0.0f;
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = 0;
#pragma unroll 1
      for (uint32_t kb = kb0; kb < kb1; kb += K_::KB_CHUNK) {
        const bool ok = pipe::wait(tfull_bar(buf), buf_phase, ctl);
        if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
        ptx::tc_fence_after();
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) {
          ptx::tmem_ld_32x32b_x32(taddr0 + buf * BN + c * 32, r);
          pipe::tmem_ld_wait32(r);
          if (c == COLS / 32 - 1) {  // in registers: the tensor core may have the buffer
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR) pipe::arrive_at(tempty0 + 8u * buf);
              else ptx::mbar_arrive(tempty0 + 8u * buf);
            }
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c * 32 + j] += __float2int_rn(__uint_as_float(r[j]));
        }
        if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
      }
      if (aborted) break;
      if (PAIR || p.split == 1) {
        const int es = p.c_dtype == SWZ_F32 ? 4 : 2;
        auto value = [&](int j) { return float(acc[j]) * (sa * sb[j]); };
        if (p.c_align >= 32 && col0 + COLS <= p.N) {
          // whole lines of C: 32 rows of 128 bytes at a time
          const int64_t r0 = row - lane + (lane / 4) * 4;
          const int64_t line = p.ldc * es;
          uint8_t* const at = static_cast<uint8_t*>(p.C) + r0 * line + col0 * es + (lane % 4) * 32;
          uint32_t o[32];
          auto put = [&](int h) {
            pipe::quad_transpose(o, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (r0 + j < p.M) pipe::st_global_32b(at + j * line + h * 128, o + 8 * j);
          };
          if (p.c_dtype == SWZ_F32) {
#pragma unroll
            for (int h = 0; h < COLS / 32; ++h) {
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(value(h * 32 + j));
              put(h);
            }
          } else {
#pragma unroll
            for (int h = 0; h < COLS / 64; ++h) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                o[j] = rows::pack16(value(h * 64 + 2 * j), value(h * 64 + 2 * j + 1), p.c_dtype);
              put(h);
            }
          }
        } else {
          // the ragged edge, and rows of C that start anywhere: a lane a column, so
          // that a store is one piece of a row
#pragma unroll
          for (int c = 0; c < COLS / 32; ++c) {
            if (col0 + c * 32 >= p.N) break;
            float f[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = value(c * 32 + j);
            pipe::transpose32(f, lane);
            const int64_t n = col0 + c * 32 + lane, r0 = row - lane;
            if (n < p.N)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (r0 + i < p.M)
                  rows::store1(static_cast<uint8_t*>(p.C) + ((r0 + i) * p.ldc + n) * es, f[i],
                               p.c_dtype);
            __syncwarp();
          }
        }
      } else if constexpr (!PAIR) {
        // partial tile to shared memory, over the ring (every load has been
        // consumed): row r, 16-byte chunk c at r * BN * 4 + (c ^ (r mod 32)) * 16
        const uint32_t r = q * 32 + lane;
#pragma unroll
        for (int c = 0; c < COLS / 4; ++c) {
          const uint32_t chunk = (part * (COLS / 4) + c) ^ (r & 31u);
          *reinterpret_cast<int4*>(smem + r * (BN * 4) + chunk * 16) =
              make_int4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
        }
      }
    }
  }

  if (!PAIR && p.split > 1) {
    // add the partial tiles: rank r of S takes rows r * 128 / S .. of the tile
    __syncwarp();
    ptx::cluster_sync();
    if (warp < kMath && !aborted) {
      const TileCoord t = tile_of(p.order, w0, p.sched_m, p.sched_n, p.group);
      const int64_t n = int64_t(t.n) * BN + lane * 4;
      const int es = p.c_dtype == SWZ_F32 ? 4 : 2;
      float sb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sb[e] = n + e < p.N ? p.sb[n + e] : 0.0f;
      auto reduce = [&](auto ranks) {
        constexpr uint32_t S = decltype(ranks)::value, RW = 8 / S, rws = 128 / S;
#pragma unroll 1
        for (uint32_t i = warp * RW; i < rws; i += kMath * RW) {
          int32_t f[RW][S][4];  // eight remote reads in flight a warp
#pragma unroll
          for (uint32_t k = 0; k < RW; ++k) {
            const uint32_t r = crank * rws + i + k;
            const uint32_t at = sA + r * (BN * 4) + ((lane ^ (r & 31u)) << 4);
#pragma unroll
            for (uint32_t j = 0; j < S; ++j)
              asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(f[k][j][0]), "=r"(f[k][j][1]), "=r"(f[k][j][2]),
                             "=r"(f[k][j][3])
                           : "r"(ptx::map_to_rank(at, j)));
          }
#pragma unroll
          for (uint32_t k = 0; k < RW; ++k) {
            const int64_t row = int64_t(t.m) * 128 + crank * rws + i + k;
            if (row >= p.M) continue;
            const float sa = p.sa[row];
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              int32_t s = f[k][0][e];
#pragma unroll
              for (uint32_t j = 1; j < S; ++j) s += f[k][j][e];
              v[e] = float(s) * (sa * sb[e]);
            }
            uint8_t* const o = static_cast<uint8_t*>(p.C) + (row * p.ldc + n) * es;
            if (n + 4 <= p.N && p.c_align >= 16) {
              if (p.c_dtype == SWZ_F32)
                *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
              else
                *reinterpret_cast<uint2*>(o) = make_uint2(rows::pack16(v[0], v[1], p.c_dtype),
                                                          rows::pack16(v[2], v[3], p.c_dtype));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n + e < p.N) rows::store1(o + e * es, v[e], p.c_dtype);
            }
          }
        }
      };
      if (p.split == 2) reduce(std::integral_constant<uint32_t, 2>{});
      else if (p.split == 4) reduce(std::integral_constant<uint32_t, 4>{});
      else reduce(std::integral_constant<uint32_t, 8>{});
    }
    __syncwarp();
    ptx::cluster_sync();  // no CTA leaves while its partial tile is read
  }

  // ---------------- teardown ----------------
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp == kMath + 1) ptx::tmem_dealloc<CG>(tmem_base, 512);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <bool PAIR>
static int launch(const CUtensorMap& ta, const CUtensorMap& tb, const Params& prm,
                  uint32_t programs, cudaStream_t stream) {
  using K_ = Cfg<PAIR>;
  auto kern = gemm_int8_kernel<PAIR>;
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  SWZ_CUDA_TRY(cudaGetDevice(&dev));
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      SWZ_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        K_::SMEM_BYTES));
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(programs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = K_::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PAIR ? 2 : prm.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, ta, tb, prm));
  return SWZ_OK;
}

static int launch_widen(const WidenArgs& a, int num_sms, cudaStream_t stream) {
  const uint64_t parts = (uint64_t(a.K) + kPart - 1) / kPart;
  const uint64_t blocks = ((uint64_t(a.rows[0]) + uint64_t(a.rows[1])) * parts + 7) / 8;
  const uint64_t cap = uint64_t(num_sms) * 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(uint32_t(blocks < cap ? blocks : cap));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, widen_kernel, a));
  return SWZ_OK;
}

struct Choice {
  int tile;        // 128: one CTA, 256: CTA pair
  uint32_t split;  // CTAs that share a tile's K (tile 128)
};

static uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// The variant with the least estimated time, in SM cycles: waves of tiles times
// (K in blocks of 64 times the cycles of one, plus a tile's fixed part).
static Choice choose(uint64_t M, uint64_t N, uint64_t K, uint32_t sms) {
  const uint64_t kb = ceil_div(K, 64);
  uint64_t best = ceil_div(ceil_div(M, 256) * ceil_div(N, 256), sms / 2) * (kb * 560 + 7000);
  Choice c{256, 1};
  const uint64_t tiles = ceil_div(M, 128) * ceil_div(N, 128);
  for (uint32_t s = 1; s <= 8; s *= 2) {
    if (s > 1 && kb < 4 * s) break;
    const uint64_t t =
        ceil_div(tiles * s, sms) * (ceil_div(kb, s) * 330 + 6000 + (s > 1 ? 3200 : 0));
    if (t < best) {
      best = t;
      c = Choice{128, s};
    }
  }
  return c;
}

// workspace: A, then (wide form) B, as fp16 in rows of whole 128-byte lines
static int64_t wide_ld(int K) { return (int64_t(K) + 63) / 64 * 64; }
static uint64_t a_bytes_of(int M, int K) { return uint64_t(M) * uint64_t(wide_ld(K)) * 2; }
static uint64_t timeout_of(const swz_gemm_int8_opts& o) {
  return uint64_t(o.timeout_ms ? o.timeout_ms : 2000u) * 1000000ull;
}

// C = A B^T of widened operands; the rest is checked.
static int product(const void* a16, const void* b16, int64_t ld, const float* sa, const float* sb,
                   void* C, int64_t ldc, int c_dtype, int M, int N, int K,
                   const swz_gemm_int8_opts& o, const DeviceInfo& dev, cudaStream_t s) {
  Choice ch = choose(uint64_t(M), uint64_t(N), uint64_t(K), uint32_t(dev.num_sms));
  if (o.tile == 256) ch = Choice{256, 1};
  if (o.tile == 128)
    ch = Choice{128, o.split_k ? uint32_t(o.split_k) : (ch.tile == 128 ? ch.split : 1u)};
  if (o.tile == 0 && o.split_k)
    ch = Choice{o.split_k == 1 ? ch.tile : 128, uint32_t(o.split_k)};
  const bool pair = ch.tile == 256;
  const uint32_t kb = uint32_t(ceil_div(uint64_t(K), pair ? 64 : 128));
  if (ch.split > kb) return SWZ_EUNSUPPORTED;  // an empty range of K
  const uint64_t sm = ceil_div(uint64_t(M), pair ? 256 : 128);
  const uint64_t sn = ceil_div(uint64_t(N), pair ? 256 : 128);
  const uint64_t cl = pair ? 2 : ch.split;
  if (sm * sn * cl > uint64_t(INT32_MAX)) return SWZ_EINVAL;
  if ((o.order == SWZ_MORTON || o.order == SWZ_XOR) &&
      !order_is_bijective(o.order, uint32_t(sm), uint32_t(sn), 1))
    return SWZ_ENOTBIJECTIVE;
  CUtensorMap ta, tb;
  int rc = encode_half(&ta, a16, 1, uint64_t(M), uint64_t(K), uint64_t(ld),
                       uint64_t(M) * uint64_t(ld), 64, 128);
  if (rc != SWZ_OK) return rc;
  rc = encode_half(&tb, b16, 1, uint64_t(N), uint64_t(K), uint64_t(ld),
                   uint64_t(N) * uint64_t(ld), 64, 128);
  if (rc != SWZ_OK) return rc;
  Params prm{};
  prm.C = C;
  prm.ldc = ldc;
  prm.sa = sa;
  prm.sb = sb;
  prm.M = M;
  prm.N = N;
  prm.c_dtype = c_dtype;
  prm.order = o.order;
  prm.group = order_uses_group(o.order) ? uint32_t(o.group) : 1u;
  prm.sched_m = uint32_t(sm);
  prm.sched_n = uint32_t(sn);
  prm.num_kb = kb;
  prm.idesc = pipe::idesc(0, 0, false, false, pair ? 256 : 128, pair ? 256 : 128);
  prm.split = ch.split;
  const uintptr_t es = c_dtype == SWZ_F32 ? 4 : 2;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(C) | (M > 1 ? uintptr_t(ldc) * es : 0);
  prm.c_align = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;
  prm.debug_flags = o.debug_flags;
  prm.timeout_ns = timeout_of(o);
  rc = op_status_word(&prm.status);
  if (rc != SWZ_OK) return rc;
  uint64_t programs = sm * sn * cl;
  if (ch.split == 1) {
    const uint64_t cap = uint64_t(dev.num_sms) / cl * cl;
    if (programs > cap) programs = cap;
  }
  return pair ? launch<true>(ta, tb, prm, uint32_t(programs), s)
              : launch<false>(ta, tb, prm, uint32_t(programs), s);
}

// How a product is made: by dp4a (few tokens), with B widened on its way to the tensor
// core (batches), or with both operands widened first.
enum Form { kTokenForm, kRingForm, kBatchForm, kWideForm };
static Form form_of(int M, int N, int K, int tile, int split) {
  if (tile == 128 || tile == 256) return kWideForm;
  // (the tokens' form reads whole pieces of 16 bytes of a row of B)
  if (tile == 0 && M <= kTokens && K >= 16) return kTokenForm;
  if (tile == 32 || (tile == 0 && M <= kRingRows)) return kRingForm;
  // (where it has the split that was asked for: how many SMs there are does not matter to that)
  if (tile == 64 || (M <= kBatchRows && batch_plan(M, N, K, split, 1).split)) return kBatchForm;
  return kWideForm;
}

static uint64_t gemm_bytes(Form f, int M, int N, int K) {
  return f == kTokenForm || f == kRingForm ? 0 : a_bytes_of(M, K) + (f == kWideForm ? a_bytes_of(N, K) : 0);
}

static int check_opts(const swz_gemm_int8_opts& o) {
  if (!order_is_valid(o.order) || (order_uses_group(o.order) && o.group < 1)) return SWZ_EINVAL;
  if (o.tile != 0 && o.tile != 32 && o.tile != 64 && o.tile != 128 && o.tile != 256) return SWZ_EUNSUPPORTED;
  if (o.split_k != 0 && o.split_k != 1 && o.split_k != 2 && o.split_k != 4 && o.split_k != 8)
    return SWZ_EUNSUPPORTED;
  if (o.tile == 256 && o.split_k > 1) return SWZ_EUNSUPPORTED;
  return SWZ_OK;
}

static int zero_result(void* C, int64_t ldc, int c_dtype, int M, int N, cudaStream_t s) {
  const int64_t es = c_dtype == SWZ_F32 ? 4 : 2;
  SWZ_CUDA_TRY(cudaMemset2DAsync(C, size_t(ldc * es), 0, size_t(N) * es, size_t(M), s));
  return SWZ_OK;
}

static bool int8_rows_ok(const void* data, int64_t ld, const float* scales, int K) {
  return data && aligned16(data) && ld >= K && ld % 16 == 0 && scales && aligned4(scales);
}

static bool result_ok(const void* C, int64_t ldc, int c_dtype, int M, int N) {
  const uintptr_t es = c_dtype == SWZ_F32 ? 4 : 2;
  return C && reinterpret_cast<uintptr_t>(C) % es == 0 && (M <= 1 || ldc >= N);
}

static RowsInMemory matrix_at(const void* p, int64_t rows, int64_t ld, int64_t width) {
  return RowsInMemory{p, rows, rows > 1 ? ld : width, width};
}
static RowsInMemory result_at(const void* C, int64_t ldc, int c_dtype, int M, int N) {
  const int64_t es = c_dtype == SWZ_F32 ? 4 : 2;
  return matrix_at(C, M, ldc * es, int64_t(N) * es);
}

// Whether a result lies over 8-bit rows or their scales, which are read while it is written.
static bool over_int8_rows(const RowsInMemory& C, const void* data, int64_t ld, const float* scales,
                           int rows, int K) {
  return rows_meet(C, matrix_at(data, rows, ld, K)) ||
         rows_meet(C, matrix_at(scales, 1, 0, int64_t(rows) * 4));
}

static bool float_type(int d) { return d == SWZ_F16 || d == SWZ_BF16 || d == SWZ_F32; }

}  // namespace i8
}  // namespace swz

using namespace swz;
using namespace swz::i8;

// A and B (either may be NULL) to fp16 in the workspace.
static int widen(const void* A, int64_t lda, int M, const void* B, int64_t ldb, int N, int K,
                 uint8_t* ws, int num_sms, cudaStream_t s) {
  WidenArgs w{};
  w.in[0] = static_cast<const uint8_t*>(A);
  w.in[1] = static_cast<const uint8_t*>(B);
  w.ld[0] = lda;
  w.ld[1] = ldb;
  w.out[0] = ws;
  w.out[1] = ws + a_bytes_of(M, K);
  w.ldo = wide_ld(K) * 2;
  w.rows[0] = A ? M : 0;
  w.rows[1] = B ? N : 0;
  w.K = K;
  return launch_widen(w, num_sms, s);
}

extern "C" int swz_gemm_int8_workspace_size_ex(int M, int N, int K, const swz_gemm_int8_opts* opts,
                                               uint64_t* h_bytes) {
  if (!h_bytes || M < 0 || N < 0 || K < 0 || K > kMaxK) return SWZ_EINVAL;
  *h_bytes = 0;
  if (M == 0 || N == 0 || K == 0) return SWZ_OK;
  *h_bytes = gemm_bytes(form_of(M, N, K, opts ? opts->tile : 0, opts ? opts->split_k : 0), M, N, K);
  return SWZ_OK;
}

extern "C" int swz_gemm_int8_workspace_size(int M, int N, int K, int tile, uint64_t* h_bytes) {
  swz_gemm_int8_opts o = {};
  o.tile = tile;
  return swz_gemm_int8_workspace_size_ex(M, N, K, &o, h_bytes);
}

extern "C" int swz_gemm_int8(const void* A, int64_t lda, const float* sa, const void* B,
                             int64_t ldb, const float* sb, void* C, int64_t ldc, int c_dtype,
                             int M, int N, int K, const swz_gemm_int8_opts* opts,
                             void* d_workspace, uint64_t workspace_bytes, void* stream) {
  swz_gemm_int8_opts o = {};
  o.order = SWZ_SERPENTINE;
  o.group = 8;
  if (opts) o = *opts;
  if (M < 0 || N < 0 || K < 0 || K > kMaxK || !float_type(c_dtype)) return SWZ_EINVAL;
  int rc = check_opts(o);
  if (rc != SWZ_OK) return rc;
  if (M == 0 || N == 0) return SWZ_OK;
  if (!result_ok(C, ldc, c_dtype, M, N)) return SWZ_EINVAL;
  if (K > 0 && (!int8_rows_ok(A, lda, sa, K) || !int8_rows_ok(B, ldb, sb, K))) return SWZ_EINVAL;
  const RowsInMemory result = result_at(C, ldc, c_dtype, M, N);
  if (K > 0 && (over_int8_rows(result, A, lda, sa, M, K) || over_int8_rows(result, B, ldb, sb, N, K)))
    return SWZ_EINVAL;
  const Form f = form_of(M, N, K, o.tile, o.split_k);
  if ((f == kTokenForm && o.split_k > 1) || (f == kRingForm && M > kRingRows))
    return SWZ_EUNSUPPORTED;
  const uint64_t need = K > 0 ? gemm_bytes(f, M, N, K) : 0;
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  if (need && (!ws || !aligned16(ws) || workspace_bytes < need)) return SWZ_EINVAL;
  DeviceInfo dev{};
  rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ldc = M > 1 ? ldc : N;
  if (K == 0) return zero_result(C, ldc, c_dtype, M, N, s);
  if (f == kTokenForm)
    return gemm_int8_tokens(A, lda, sa, nullptr, 0, 0, B, ldb, sb, C, ldc, c_dtype, M, N, K,
                            dev.num_sms, s);
  if (f == kRingForm)
    return gemm_int8_rows(A, lda, sa, B, ldb, sb, C, ldc, c_dtype, M, N, K, o.split_k,
                          o.debug_flags, timeout_of(o), false, dev.num_sms, s);
  BatchPlan b{};
  if (f == kBatchForm) {
    b = batch_plan(M, N, K, o.split_k, dev.num_sms);
    if (!b.split) return SWZ_EUNSUPPORTED;
  }
  rc = widen(A, lda, M, f == kWideForm ? B : nullptr, ldb, N, K, ws, dev.num_sms, s);
  if (rc != SWZ_OK) return rc;
  if (f == kBatchForm)
    return gemm_int8_batch(ws, wide_ld(K), sa, B, ldb, sb, C, ldc, c_dtype, M, N, K, b,
                           o.debug_flags, timeout_of(o), s);
  return product(ws, ws + a_bytes_of(M, K), wide_ld(K), sa, sb, C, ldc, c_dtype, M, N, K, o, dev,
                 s);
}

// workspace of the layer: the scales of x, then x as bytes (few tokens that not every CTA
// quantises itself) or what the product has
static uint64_t linear_scales_bytes(int M) { return (uint64_t(M) * 4 + 255) & ~uint64_t(255); }
static int64_t bytes_ld(int K) { return (int64_t(K) + 15) / 16 * 16; }
static uint64_t linear_bytes(Form f, bool fused, int M, int N, int K) {
  if (fused) return 0;
  if (f == kTokenForm || f == kRingForm)
    return linear_scales_bytes(M) + uint64_t(M) * uint64_t(bytes_ld(K));
  return linear_scales_bytes(M) + gemm_bytes(f, M, N, K);
}

extern "C" int swz_linear_int8_workspace_size(int M, int N, int K, uint64_t* h_bytes) {
  if (!h_bytes || M < 0 || N < 0 || K < 0 || K > kMaxK) return SWZ_EINVAL;
  *h_bytes = 0;
  if (M == 0 || N == 0 || K == 0) return SWZ_OK;
  const Form f = form_of(M, N, K, 0, 0);
  *h_bytes = linear_bytes(f, f == kTokenForm && tokens_fused(M, K), M, N, K);
  return SWZ_OK;
}

extern "C" int swz_linear_int8(const void* x, int dtype, int64_t ldx, const void* W, int64_t ldw,
                               const float* sw, void* y, int64_t ldy, int y_dtype, int M, int N,
                               int K, void* d_workspace, uint64_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || K > kMaxK || !float_type(dtype) || !float_type(y_dtype))
    return SWZ_EINVAL;
  if (M == 0 || N == 0) return SWZ_OK;
  const uintptr_t es = dtype == SWZ_F32 ? 4 : 2;
  if (!result_ok(y, ldy, y_dtype, M, N)) return SWZ_EINVAL;
  if (K > 0 && (!x || reinterpret_cast<uintptr_t>(x) % es != 0 || (M > 1 && ldx < K) ||
                !int8_rows_ok(W, ldw, sw, K)))
    return SWZ_EINVAL;
  const RowsInMemory result = result_at(y, ldy, y_dtype, M, N);
  if (K > 0 && over_int8_rows(result, W, ldw, sw, N, K)) return SWZ_EINVAL;
  const Form f = form_of(M, N, K, 0, 0);
  // where every CTA quantises x itself, y must not be written over it
  const bool fused = f == kTokenForm && tokens_fused(M, K) &&
                     !rows_meet(result, matrix_at(x, M, ldx * int64_t(es), int64_t(K) * int64_t(es)));
  const uint64_t need = K > 0 ? linear_bytes(f, fused, M, N, K) : 0;
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  if (need && (!ws || !aligned16(ws) || workspace_bytes < need)) return SWZ_EINVAL;
  DeviceInfo dev{};
  int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ldy = M > 1 ? ldy : N;
  if (K == 0) return zero_result(y, ldy, y_dtype, M, N, s);
  if (fused)
    return gemm_int8_tokens(nullptr, 0, nullptr, x, dtype, ldx, W, ldw, sw, y, ldy, y_dtype, M, N,
                            K, dev.num_sms, s);
  float* sx = reinterpret_cast<float*>(ws);
  ws += linear_scales_bytes(M);
  swz_gemm_int8_opts o = {};
  o.order = SWZ_SERPENTINE;
  o.group = 8;
  if (f == kTokenForm || f == kRingForm) {
    rc = quantize_rows(x, dtype, ldx, M, K, ws, bytes_ld(K), sx, false, s);
    if (rc != SWZ_OK) return rc;
    if (f == kRingForm)
      return gemm_int8_rows(ws, bytes_ld(K), sx, W, ldw, sw, y, ldy, y_dtype, M, N, K, 0, 0,
                            timeout_of(o), true, dev.num_sms, s);
    return gemm_int8_tokens(ws, bytes_ld(K), sx, nullptr, 0, 0, W, ldw, sw, y, ldy, y_dtype, M, N,
                            K, dev.num_sms, s);
  }
  rc = quantize_rows(x, dtype, ldx, M, K, ws, wide_ld(K) * 2, sx, true, s);
  if (rc != SWZ_OK) return rc;
  if (f == kBatchForm)
    return gemm_int8_batch(ws, wide_ld(K), sx, W, ldw, sw, y, ldy, y_dtype, M, N, K,
                           batch_plan(M, N, K, 0, dev.num_sms), 0, timeout_of(o), s);
  rc = widen(nullptr, 0, M, W, ldw, N, K, ws, dev.num_sms, s);
  if (rc != SWZ_OK) return rc;
  return product(ws, ws + a_bytes_of(M, K), wide_ld(K), sx, sw, y, ldy, y_dtype, M, N, K, o, dev,
                 s);
}
