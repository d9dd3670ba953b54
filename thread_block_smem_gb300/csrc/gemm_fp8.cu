// gemm_fp8.cu -- C = A * B^T of 8-bit operands with one fp32 scale for each
// block of 128 along K:
//     C[m, n] = sum over blocks kb of  sa[m, kb] sb[n, kb]
//               * sum over k in kb of  A[m, k] B[n, k]
// A (M x K) has row blocks (1 x 128); B (N x K) square (128 x 128) or row
// blocks.  Both K-major, e4m3 or e5m2 each; C fp32, bf16 or fp16.
//
// Mathematics and split: the tensor core sums a block's 128 products in fp32;
// the sum is scaled and added to fp32 accumulators in registers.  So every
// block of K is an MMA accumulation of its own, and its tile is read back from
// TMEM, multiplied and added.
//   * One CTA per SM, 12 warps: 0-7 the sums (warp w: TMEM lanes 32 (w mod 4)
//     .., columns 64 (w / 4) .. of the tile), 8 TMA producer, 9 and 10 MMA
//     issue (9 also TMEM allocation), 11 scales.
//   * Tiles of 128 columns: TMEM holds four in turn, so the tensor core runs
//     ahead of the readers; a stage of shared memory is one block of K (128
//     bytes a row).  CTA pair: 256 x 128 (each CTA 128 rows of A and 64 of B),
//     one CTA: 128 x 128.  256-column tiles leave two TMEM buffers: a block's
//     MMAs (512 cycles) then wait for a whole hand-over, 8192^3 in 467 us
//     against 410-425.
//   * Scales go through a ring of shared memory of their own, 12 blocks deep:
//     loaded by the summing warps themselves, two blocks ahead, each block cost
//     an L2 round trip.  4-byte copies: rows of scales start anywhere.
//   * split: a cluster of 2, 4 or 8 CTAs shares one 128 x 128 tile by ranges
//     of K and adds the partial tiles through distributed shared memory in
//     rank order (deterministic, no workspace): for few tiles.
//   * tiles are dealt out by the framework's tile orders, w = cluster + i P.
//
// What bounds it: the summing warps.  A 128 x 128 tile's MMAs take 256 cycles
// a block; waits, TMEM loads, release and 64 FMAs a thread take 440 to 480, and
// 16 warps of half the columns the same.  With a quarter of the MMAs 8192^3
// takes 392 us, with half the operand traffic as well the same.  Measured at
// 8192^3, bf16 result: 410-425 us, 2.6-2.7 PFLOP/s, 0.70 of twice the measured
// bf16 peak (467 in a stream of seconds, at 1.70 GHz under the power cap); tensor
// pipe 56 % busy, issue slots 50 %.  B in row blocks 650 us: a scale a column is
// twice the arithmetic, which costs little (432 us without the reads), and 64
// registers a thread and block from shared memory, whose pipe the counters show
// busy for 46 % of the time (11 % with square blocks).  TMEM's 16-lane order reads
// a quarter of the scales, but half as many lanes at a time: 697.  The single-CTA
// kernels spill 40 bytes a thread, the pairs nothing.
#include <mutex>
#include <type_traits>

#include "common.h"
#include "f8.cuh"
#include "ops.h"
#include "pipe.cuh"
#include "tile_order.cuh"

namespace swz {
namespace gemm8 {

constexpr int BM = 128, BN = 128, BK = 128;
constexpr int kMath = 8;       // summing warps
constexpr int kIssuers = 2;    // warps that issue MMAs, a block of K each in turn
constexpr int kThreads = (kMath + 2 + kIssuers) * 32;
constexpr int kScaleKb = 4;    // blocks of K whose scales share a slot of the ring

constexpr int COLS = 4 * BN / kMath;  // columns a summing warp holds
static_assert(COLS == 64, "two TMEM loads of 32 columns");

template <bool PAIR>
struct Cfg {
  static constexpr int CG = PAIR ? 2 : 1;
  static constexpr int BN_LOCAL = BN / CG;  // rows of B this CTA loads
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN_LOCAL * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = PAIR ? 8 : 6;
  static constexpr int NBUF = 512 / BN;   // tiles of TMEM
  static constexpr int SLOTS = 3;         // ring of scales: 128 of A's rows, then B's,
  static constexpr int SLOT = BM + BN;    // floats, of kScaleKb blocks
  static constexpr int BARS = 2 * STAGES + 2 * NBUF + 2 * SLOTS + kIssuers;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + SLOTS * kScaleKb * SLOT * 4 + BARS * 8 + 16;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(STAGES % kIssuers == 0 && NBUF % kIssuers == 0, "an issuer keeps its stages");
  static_assert(STAGES * STAGE_BYTES >= BM * BN * 4, "a partial tile fits the ring");
};

struct Params {
  void* C;
  int64_t ldc;
  const float* sa;
  int64_t ldsa;
  const float* sb;
  int64_t ldsb;
  int M, N;
  int c_dtype;
  int order;
  uint32_t group, sched_m, sched_n, num_kb, idesc, split;
  uint32_t c_align;  // bytes that every row start and base of C are a multiple of (32, 16 or less)
  uint32_t debug_flags;
  unsigned int* status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ uint32_t pack_out(float a, float b, int dtype) {
  if (dtype == SWZ_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// one element, for the ragged edge and unaligned rows
__device__ __forceinline__ void store1(void* C, int64_t at, float v, int dtype) {
  if (dtype == SWZ_F32) static_cast<float*>(C)[at] = v;
  else if (dtype == SWZ_BF16) static_cast<__nv_bfloat16*>(C)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(C)[at] = __float2half_rn(v);
}

// 16 consecutive elements of a row starting at column n (a multiple of 16)
__device__ __forceinline__ void store16(const Params& p, int64_t row, int n, const float (&f)[16]) {
  const int64_t at = row * p.ldc + n;
  if (n + 16 <= p.N && p.c_align >= 16) {
    if (p.c_dtype == SWZ_F32) {
      float* c = static_cast<float*>(p.C) + at;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(f[8 * h + j]);
        if (p.c_align >= 32) {
          pipe::st_global_32b(c + 8 * h, v);
        } else {
          *reinterpret_cast<uint4*>(c + 8 * h) = make_uint4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<uint4*>(c + 8 * h + 4) = make_uint4(v[4], v[5], v[6], v[7]);
        }
      }
    } else {
      uint16_t* c = static_cast<uint16_t*>(p.C) + at;
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = pack_out(f[2 * j], f[2 * j + 1], p.c_dtype);
      if (p.c_align >= 32) {
        pipe::st_global_32b(c, v);
      } else {
        *reinterpret_cast<uint4*>(c) = make_uint4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<uint4*>(c + 8) = make_uint4(v[4], v[5], v[6], v[7]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (n + j < p.N) store1(p.C, at + j, f[j], p.c_dtype);
  }
}

template <bool PAIR, bool BROW>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA,
                    const __grid_constant__ CUtensorMap tmB, const Params p) {
  using K_ = Cfg<PAIR>;
  constexpr int CG = K_::CG, STAGES = K_::STAGES, NBUF = K_::NBUF;
  constexpr uint32_t SLOTS = K_::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sA = ptx::smem_u32(smem);
  const uint32_t sB = sA + STAGES * K_::A_BYTES;
  float* const ring = reinterpret_cast<float*>(smem + STAGES * K_::STAGE_BYTES);
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(smem + STAGES * K_::STAGE_BYTES +
                                  SLOTS * kScaleKb * K_::SLOT * 4);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * STAGES + NBUF + a); };
  auto sfull_bar = [&](uint32_t i) { return bar0 + 8u * (2 * STAGES + 2 * NBUF + i); };
  auto sempty_bar = [&](uint32_t i) { return bar0 + 8u * (2 * STAGES + 2 * NBUF + SLOTS + i); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * NBUF + 2 * SLOTS);
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
    for (uint32_t i = 0; i < SLOTS; ++i) {
      ptx::mbar_init(sfull_bar(i), 32);
      ptx::mbar_init(sempty_bar(i), kMath);
    }
    for (int i = 0; i < kIssuers; ++i) ptx::mbar_init(drain_bar + 8u * i, 1);
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
      const int32_t m0 = int32_t((t.m * CG + rank) * BM);
      const int32_t n0 = int32_t(t.n * BN + rank * K_::BN_LOCAL);
      for (uint32_t kb = kb0; kb < kb1; ++kb) {
        const bool ok = pipe::wait(empty_bar(stage), phase ^ 1u, ctl);
        if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
        if (pipe::elect_one()) {
          if (leader) ptx::mbar_arrive_expect_tx(full_bar(stage), CG * K_::STAGE_BYTES);
          if (!skip) {
            const int32_t k0 = int32_t(kb * BK);
            const uint32_t a_dst = sA + stage * K_::A_BYTES, b_dst = sB + stage * K_::B_BYTES;
            if constexpr (PAIR) {
              ptx::tma_load_2d_pair(a_dst, &tmA, full0 + 8u * stage, k0, m0, pol);
              ptx::tma_load_2d_pair(b_dst, &tmB, full0 + 8u * stage, k0, n0, pol);
            } else {
              ptx::tma_load_2d(a_dst, &tmA, full0 + 8u * stage, k0, m0, pol);
              ptx::tma_load_2d(b_dst, &tmB, full0 + 8u * stage, k0, n0, pol);
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
  } else if (warp > kMath && warp <= kMath + kIssuers) {
    // ---------------- MMA issuers (leader CTA) ----------------
    // The whole warp runs the loop and one elected lane issues: descriptors
    // then live in uniform registers.  With the loop inside one lane's branch
    // every operand of an MMA was moved there first, and the four MMAs of a
    // block took twice as long to issue as to run.
    if (leader) {
      // issuer i takes every kIssuers-th block: each is an accumulation of its
      // own, so their order does not matter, and the barrier tests and commits
      // of one pass while the other's MMAs run
      const uint32_t me = warp - (kMath + 1);
      uint32_t stage = me, phase = 0, buf = me, buf_phase = 0, turn = me;
      bool issued = false;
      const uint64_t adesc0 = pipe::sdesc128(sA, 16, 1024);
      const uint64_t bdesc0 = pipe::sdesc128(sB, 16, 1024);
      for (uint32_t w = w0; w < units && !aborted; w += P) {
        uint32_t kb = kb0 + turn;  // the first of this tile's blocks that is mine
        for (; kb < kb1; kb += kIssuers) {
          const bool ok = pipe::wait(full_bar(stage), phase, ctl) &&
                          pipe::wait(tempty_bar(buf), buf_phase ^ 1u, ctl);
          if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
          ptx::tc_fence_after();
          const uint64_t a = adesc0 + uint64_t(stage * uint32_t(K_::A_BYTES >> 4));
          const uint64_t b = bdesc0 + uint64_t(stage * uint32_t(K_::B_BYTES >> 4));
          const uint32_t d = tmem_base + buf * BN;
          if (pipe::elect_one()) {
#pragma unroll
            for (uint32_t kk = 0; kk < BK / 32; ++kk)
              pipe::mma_f8<CG>(d, a + kk * 2, b + kk * 2, p.idesc, kk != 0);
            if constexpr (PAIR) {
              ptx::mma_commit_pair(tfull_bar(buf), 0x3);
              ptx::mma_commit_pair(empty_bar(stage), 0x3);
            } else {
              ptx::mma_commit(tfull_bar(buf));
              ptx::mma_commit(empty_bar(stage));
            }
          }
          __syncwarp();
          issued = true;
          stage += kIssuers;
          if (stage >= uint32_t(STAGES)) { stage -= STAGES; phase ^= 1u; }
          buf += kIssuers;
          if (buf >= uint32_t(NBUF)) { buf -= NBUF; buf_phase ^= 1u; }
        }
        turn = kb - kb1;  // blocks of the next tile before mine
      }
      if (aborted && issued) {
        // drain: wait (bounded) until every MMA issued so far has completed
        const uint32_t drain = drain_bar + 8u * me;
        if (pipe::elect_one()) {
          if constexpr (PAIR) ptx::mma_commit_pair(drain, 0x1);
          else ptx::mma_commit(drain);
        }
        const uint64_t t0 = ptx::global_timer_ns();
        while (!pipe::try_wait(drain, 0) && ptx::global_timer_ns() - t0 < p.timeout_ns) {
        }
      }
    }
    __syncwarp();
  } else if (warp > kMath + kIssuers) {
    // ---------------- scales ----------------
    uint32_t slot = 0, phase = 0;
    const uint32_t ring0 = ptx::smem_u32(ring);
    for (uint32_t w = w0; w < units && !aborted; w += P) {
      const TileCoord t = tile_of(p.order, w, p.sched_m, p.sched_n, p.group);
      const int64_t m0 = int64_t(t.m * CG + rank) * BM + lane;
      const int64_t n0 = int64_t(t.n) * BN;
      for (uint32_t kb = kb0; kb < kb1; kb += kScaleKb) {
        const bool ok = pipe::wait(sempty_bar(slot), phase ^ 1u, ctl);
        if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
#pragma unroll 1
        for (uint32_t i = 0; i < uint32_t(kScaleKb) && kb + i < kb1; ++i) {
          const uint32_t dst = ring0 + (slot * kScaleKb + i) * (K_::SLOT * 4) + lane * 4;
          const float* sa = p.sa + int64_t(kb + i) * p.ldsa;
#pragma unroll
          for (int j = 0; j < BM / 32; ++j)
            pipe::copy4(dst + j * 128, sa + m0 + j * 32, m0 + j * 32 < p.M, p.sa);
          if constexpr (BROW) {
            const float* sb = p.sb + int64_t(kb + i) * p.ldsb;
            const int64_t n = n0 + lane;
#pragma unroll
            for (int j = 0; j < BN / 32; ++j)
              pipe::copy4(dst + (BM + j * 32) * 4, sb + n + j * 32, n + j * 32 < p.N, p.sb);
          } else if (lane < uint32_t(BN / 128)) {  // the tile's square blocks
            const int64_t n = n0 + lane * 128;
            pipe::copy4(dst + BM * 4, p.sb + n / 128 * p.ldsb + kb + i, n < p.N, p.sb);
          }
        }
        pipe::copies_arrive(sfull_bar(slot));
        if (++slot == SLOTS) { slot = 0; phase ^= 1u; }
      }
    }
    pipe::copies_wait();
    __syncwarp();
  } else {
    // ---------------- sums ----------------
    const uint32_t q = warp & 3u, part = warp >> 2;  // rows 32 q .., columns COLS part ..
    uint32_t buf = 0, buf_phase = 0, slot = 0, slot_phase = 0;
    const uint32_t tfull0 = tfull_bar(0), sfull0 = sfull_bar(0), sempty0 = sempty_bar(0);
    const uint32_t tempty0 = PAIR ? ptx::map_to_rank(tempty_bar(0), 0) : tempty_bar(0);
    const uint32_t taddr0 = tmem_base + ((q * 32u) << 16) + part * COLS;
    // this thread's row scale, and its warp's scales of B, in the ring's first block
    const uint32_t sa0 = ptx::smem_u32(ring) + (q * 32 + lane) * 4;
    const uint32_t sb_off = BROW ? (BM + part * COLS - (q * 32 + lane)) * 4
                                 : (BM + part * COLS / 128 - (q * 32 + lane)) * 4;
    uint64_t acc[COLS / 2];
    uint32_t r[2][32];  // the block's columns, as two halves
    auto add = [&](uint32_t(&d)[32], int c, float s, uint32_t sa) {
      const uint64_t s2 = pipe::pack2(s, s);
      if constexpr (BROW) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float b[4];
          pipe::ld_shared4(sa + sb_off + (c * 32 + 4 * j) * 4, b);
          uint64_t* a = acc + c * 16 + 2 * j;
          a[0] = pipe::fma2(pipe::pack2(d[4 * j], d[4 * j + 1]),
                            pipe::mul2(pipe::pack2(b[0], b[1]), s2), a[0]);
          a[1] = pipe::fma2(pipe::pack2(d[4 * j + 2], d[4 * j + 3]),
                            pipe::mul2(pipe::pack2(b[2], b[3]), s2), a[1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          acc[c * 16 + j] = pipe::fma2(pipe::pack2(d[2 * j], d[2 * j + 1]), s2, acc[c * 16 + j]);
      }
    };
    // scales of the block at `sa`
    auto scale = [&](uint32_t sa) {
      float s = pipe::ld_shared(sa);
      if constexpr (!BROW) s *= pipe::ld_shared(sa + sb_off);
      return s;
    };
    // The scales' slot of the next block, at the start of one.  One vote for
    // its four blocks: after a wait that ran out the next ones return at once
    // (the abort flag), and what is summed is not used.
    auto take_slot = [&]() {
      const bool ok = pipe::wait(sfull0 + 8u * slot, slot_phase, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok && *ctl.abort_flag == 0)) aborted = true;
      const uint32_t sa = sa0 + slot * (kScaleKb * K_::SLOT * 4);
      if (++slot == SLOTS) { slot = 0; slot_phase ^= 1u; }
      return sa;
    };
    auto free_slot = [&]() {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(sempty0 + 8u * (slot == 0 ? SLOTS - 1 : slot - 1));
    };
    // both halves are in registers: the tensor core may have the buffer
    auto landed = [&]() {
      pipe::tmem_ld_wait32(r[0]);
      pipe::tmem_ld_wait32(r[1]);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) pipe::arrive_at(tempty0 + 8u * buf);
        else ptx::mbar_arrive(tempty0 + 8u * buf);
      }
      if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
    };
    for (uint32_t w = w0; w < units && !aborted; w += P) {
      const TileCoord t = tile_of(p.order, w, p.sched_m, p.sched_n, p.group);
      const int64_t row = int64_t(t.m * CG + rank) * BM + q * 32 + lane;
      const int64_t col0 = int64_t(t.n) * BN + part * COLS;
      const bool row_in = row < p.M;
#pragma unroll
      for (int j = 0; j < COLS / 2; ++j) acc[j] = 0ull;
      uint32_t sa = take_slot();
      pipe::wait(tfull0 + 8u * buf, buf_phase, ctl);
      __syncwarp();
      ptx::tc_fence_after();
      ptx::tmem_ld_32x32b_x32(taddr0 + buf * BN, r[0]);
      ptx::tmem_ld_32x32b_x32(taddr0 + buf * BN + 32, r[1]);
      float s = scale(sa);
      landed();
      // The next block's barrier is tested and its first half loaded between
      // the two halves of this one: with a block's wait, loads, release and
      // 64 FMAs one after the other a warp took 500 cycles for a block, and
      // twice the warps took as long.
#pragma unroll 1
      for (uint32_t kb = kb0 + 1; kb < kb1 && !aborted; ++kb) {
        const bool ready = pipe::test_wait(tfull0 + 8u * buf, buf_phase);
        add(r[0], 0, s, sa);
        const bool turn = (kb - kb0) % kScaleKb == 0;
        const uint32_t sa_cur = sa;
        const float s_cur = s;
        if (!ready) pipe::wait(tfull0 + 8u * buf, buf_phase, ctl);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_ld_32x32b_x32(taddr0 + buf * BN, r[0]);
        add(r[1], 1, s_cur, sa_cur);
        if (turn) {
          free_slot();
          sa = take_slot();
        } else {
          sa += K_::SLOT * 4;
        }
        ptx::tmem_ld_32x32b_x32(taddr0 + buf * BN + 32, r[1]);
        s = scale(sa);
        landed();
      }
      add(r[0], 0, s, sa);
      add(r[1], 1, s, sa);
      free_slot();
      if (aborted) break;
      if (PAIR || p.split == 1) {
        if ((BROW || !PAIR) && p.c_align >= 32 && col0 + COLS <= p.N) {
          // Whole lines of C: 32 rows of 128 bytes (one of 16-bit values, two
          // of fp32) at a time.  2 to 5 % of 8192^3; the pair with square blocks,
          // whose sums' loop it leaves fewer registers, is 5 % slower with it.
          static_assert(COLS == 64, "a row of 16-bit results is 128 bytes");
          const int64_t r0 = row - lane + (lane / 4) * 4;
          const int parts = p.c_dtype == SWZ_F32 ? 2 : 1;
          const int64_t line = p.ldc * (p.c_dtype == SWZ_F32 ? 4 : 2);
          uint8_t* const at = static_cast<uint8_t*>(p.C) + r0 * line +
                              col0 * (p.c_dtype == SWZ_F32 ? 4 : 2) + (lane % 4) * 32;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h >= parts) break;
            uint32_t o[32];
            if (p.c_dtype == SWZ_F32) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float a, b;
                pipe::unpack2(acc[h * 16 + j], a, b);
                o[2 * j] = __float_as_uint(a);
                o[2 * j + 1] = __float_as_uint(b);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                float a, b;
                pipe::unpack2(acc[j], a, b);
                o[j] = pack_out(a, b, p.c_dtype);
              }
            }
            pipe::quad_transpose(o, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (r0 + j < p.M) pipe::st_global_32b(at + j * line + h * 128, o + 8 * j);
          }
        } else if (p.c_align >= 16) {
#pragma unroll
          for (int c = 0; c < COLS / 16; ++c) {
            const int64_t n = col0 + c * 16;
            if (n >= p.N) break;
            float f[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) pipe::unpack2(acc[c * 8 + j], f[2 * j], f[2 * j + 1]);
            if (row_in) store16(p, row, int(n), f);
          }
        } else {
          // rows of C that start anywhere: a lane a column instead of a row, so
          // that a store is one piece of a row (element by element from the
          // rows' lanes it took 5 times as long)
#pragma unroll
          for (int c = 0; c < COLS / 32; ++c) {
            float f[32];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              pipe::unpack2(acc[c * 16 + j], f[2 * j], f[2 * j + 1]);
            pipe::transpose32(f, lane);
            const int64_t n = col0 + c * 32 + lane, r0 = row - lane;
            if (n < p.N)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (r0 + i < p.M) store1(p.C, (r0 + i) * p.ldc + n, f[i], p.c_dtype);
            __syncwarp();
          }
        }
      } else {
        // partial tile to shared memory, over the ring (every load has been
        // consumed): row r, 16-byte chunk c at r * BN * 4 + (c ^ (r mod 32)) * 16
        const uint32_t r = q * 32 + lane;
#pragma unroll
        for (int c = 0; c < COLS / 4; ++c) {
          float a, b, d, e;
          pipe::unpack2(acc[2 * c], a, b);
          pipe::unpack2(acc[2 * c + 1], d, e);
          const uint32_t chunk = (part * (COLS / 4) + c) ^ (r & 31u);
          *reinterpret_cast<float4*>(smem + r * (BN * 4) + chunk * 16) = make_float4(a, b, d, e);
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
      // A remote read takes about 1 us: a warp has eight of them in flight,
      // from all S ranks for 8 / S rows.
      auto reduce = [&](auto ranks) {
        constexpr uint32_t S = decltype(ranks)::value, RW = 8 / S, rows = BM / S;
#pragma unroll 1
        for (uint32_t i = warp * RW; i < rows; i += kMath * RW) {
          float f[RW][S][4];
#pragma unroll
          for (uint32_t k = 0; k < RW; ++k) {
            const uint32_t r = crank * rows + i + k;
            const uint32_t at = sA + r * (BN * 4) + ((lane ^ (r & 31u)) << 4);
#pragma unroll
            for (uint32_t j = 0; j < S; ++j)
              asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(f[k][j][0]), "=f"(f[k][j][1]), "=f"(f[k][j][2]),
                             "=f"(f[k][j][3])
                           : "r"(ptx::map_to_rank(at, j)));
          }
#pragma unroll
          for (uint32_t k = 0; k < RW; ++k) {
            const int64_t row = int64_t(t.m) * BM + crank * rows + i + k;
            if (row >= p.M) continue;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[e] = f[k][0][e];
#pragma unroll
              for (uint32_t j = 1; j < S; ++j) v[e] += f[k][j][e];
            }
            const int64_t o = row * p.ldc + n;
            if (n + 4 <= p.N && p.c_align >= 16) {
              if (p.c_dtype == SWZ_F32)
                *reinterpret_cast<float4*>(static_cast<float*>(p.C) + o) =
                    make_float4(v[0], v[1], v[2], v[3]);
              else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + o) = make_uint2(
                    pack_out(v[0], v[1], p.c_dtype), pack_out(v[2], v[3], p.c_dtype));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n + e < p.N) store1(p.C, o + e, v[e], p.c_dtype);
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
template <bool PAIR, bool BROW>
static int launch(const CUtensorMap& ta, const CUtensorMap& tb, const Params& prm,
                  uint32_t programs, cudaStream_t stream) {
  using K_ = Cfg<PAIR>;
  auto kern = gemm_fp8_kernel<PAIR, BROW>;
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

struct Choice {
  int tile;        // 128: one CTA, 256: CTA pair
  uint32_t split;  // CTAs that share a tile's K (tile 128)
};

static uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// The variant with the least estimated time, in SM cycles: waves of tiles
// times (blocks of K times the cycles of one, plus a tile's fixed part), fitted
// to one to four waves of 4096 x 4096 and to splits of 27 to 256 tiles.
static Choice choose(uint64_t M, uint64_t N, uint64_t kb, uint32_t sms) {
  const uint64_t pairs = sms / 2, tn = ceil_div(N, 128);
  uint64_t best = ceil_div(ceil_div(M, 256) * tn, pairs) * (kb * 370 + 5800);
  Choice c{256, 1};
  const uint64_t tiles = ceil_div(M, 128) * tn;
  for (uint32_t s = 1; s <= 8; s *= 2) {
    if (s > 1 && kb < 2 * s) break;
    const uint64_t t =
        ceil_div(tiles * s, sms) * (ceil_div(kb, s) * 390 + 6200 + (s > 1 ? 3200 : 0));
    if (t < best) {
      best = t;
      c = Choice{128, s};
    }
  }
  return c;
}

}  // namespace gemm8
}  // namespace swz

using namespace swz;
using namespace swz::gemm8;

static bool matrix_ok(const swz_fp8_matrix* m, int rows, int K) {
  const int64_t kb = (int64_t(K) + 127) / 128;
  return m->data && aligned16(m->data) && m->ld >= K && m->ld % 16 == 0 && m->scales &&
         aligned4(m->scales) && m->ld_scales >= (m->block == SWZ_BLOCK_SQUARE ? kb : int64_t(rows));
}

extern "C" int swz_gemm_fp8(const swz_fp8_matrix* A, const swz_fp8_matrix* B, void* C, int64_t ldc,
                            int c_dtype, int M, int N, int K, const swz_gemm_fp8_opts* opts,
                            void* stream) {
  return swz::gemm_fp8(A, B, C, ldc, c_dtype, M, N, K, opts, stream, false);
}

int swz::gemm_fp8(const swz_fp8_matrix* A, const swz_fp8_matrix* B, void* C, int64_t ldc,
                  int c_dtype, int M, int N, int K, const swz_gemm_fp8_opts* opts, void* stream,
                  bool early_b) {
  swz_gemm_fp8_opts o = {};
  o.order = SWZ_SERPENTINE;
  o.group = 8;
  if (opts) o = *opts;
  if (M < 0 || N < 0 || K < 0 || !A || !B) return SWZ_EINVAL;
  if (!order_is_valid(o.order) || (order_uses_group(o.order) && o.group < 1)) return SWZ_EINVAL;
  if (c_dtype != SWZ_F16 && c_dtype != SWZ_BF16 && c_dtype != SWZ_F32) return SWZ_EINVAL;
  for (const swz_fp8_matrix* m : {A, B}) {
    if (m->fmt != SWZ_E4M3 && m->fmt != SWZ_E5M2) return SWZ_EINVAL;
    if (m->block != SWZ_BLOCK_ROW && m->block != SWZ_BLOCK_SQUARE) return SWZ_EINVAL;
  }
  if (A->block != SWZ_BLOCK_ROW) return SWZ_EUNSUPPORTED;
  if (o.tile != 0 && o.tile != 128 && o.tile != 256) return SWZ_EUNSUPPORTED;
  if (o.split_k != 0 && o.split_k != 1 && o.split_k != 2 && o.split_k != 4 && o.split_k != 8)
    return SWZ_EUNSUPPORTED;
  if (o.tile == 256 && o.split_k > 1) return SWZ_EUNSUPPORTED;
  if (o.num_programs < 0 || (o.num_programs && o.tile == 0)) return SWZ_EINVAL;
  if (M == 0 || N == 0) return SWZ_OK;
  const int64_t es = c_dtype == SWZ_F32 ? 4 : 2;
  const uintptr_t ca = reinterpret_cast<uintptr_t>(C);
  if (!C || ca % uintptr_t(es) != 0 || (M > 1 && ldc < N)) return SWZ_EINVAL;
  if (K > 0 && (!matrix_ok(A, M, K) || !matrix_ok(B, N, K))) return SWZ_EINVAL;
  DeviceInfo dev{};
  int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t ld = M > 1 ? ldc : N;
  if (K == 0) {
    SWZ_CUDA_TRY(cudaMemset2DAsync(C, size_t(ld * es), 0, size_t(N) * es, size_t(M), s));
    return SWZ_OK;
  }
  const uint32_t kb = uint32_t((int64_t(K) + 127) / 128);
  const uint64_t timeout_ns = uint64_t(o.timeout_ms ? o.timeout_ms : 2000u) * 1000000ull;
  if (o.tile == 0 && M <= kFewRows) {
    if (o.split_k > 0 && uint32_t(o.split_k) > kb) return SWZ_EUNSUPPORTED;
    return gemm_fp8_rows(*A, *B, C, ld, c_dtype, M, N, K, o.split_k, o.debug_flags, timeout_ns,
                         early_b, dev.num_sms, s);
  }
  Choice ch = choose(uint64_t(M), uint64_t(N), kb, uint32_t(dev.num_sms));
  if (o.tile == 256) ch = Choice{256, 1};
  if (o.tile == 128) ch = Choice{128, o.split_k ? uint32_t(o.split_k) : (ch.tile == 128 ? ch.split : 1u)};
  if (o.tile == 0 && o.split_k) ch = Choice{o.split_k == 1 ? ch.tile : 128, uint32_t(o.split_k)};
  if (ch.split > kb) return SWZ_EUNSUPPORTED;  // an empty range of K
  const bool pair = ch.tile == 256;
  const uint64_t sm = ceil_div(uint64_t(M), pair ? 256 : 128);
  const uint64_t sn = ceil_div(uint64_t(N), BN);
  const uint64_t cl = pair ? 2 : ch.split;
  if (sm * sn * cl > uint64_t(INT32_MAX)) return SWZ_EINVAL;
  if ((o.order == SWZ_MORTON || o.order == SWZ_XOR) &&
      !order_is_bijective(o.order, uint32_t(sm), uint32_t(sn), 1))
    return SWZ_ENOTBIJECTIVE;
  if (o.num_programs % int(cl) != 0) return SWZ_EINVAL;

  CUtensorMap ta, tb;
  rc = encode_bytes(&ta, A->data, uint64_t(M), uint64_t(K), uint64_t(A->ld), 128);
  if (rc != SWZ_OK) return rc;
  rc = encode_bytes(&tb, B->data, uint64_t(N), uint64_t(K), uint64_t(B->ld), pair ? 64 : 128);
  if (rc != SWZ_OK) return rc;

  Params prm{};
  prm.C = C;
  prm.ldc = ld;
  prm.sa = A->scales;
  prm.ldsa = A->ld_scales;
  prm.sb = B->scales;
  prm.ldsb = B->ld_scales;
  prm.M = M;
  prm.N = N;
  prm.c_dtype = c_dtype;
  prm.order = o.order;
  prm.group = order_uses_group(o.order) ? uint32_t(o.group) : 1u;
  prm.sched_m = uint32_t(sm);
  prm.sched_n = uint32_t(sn);
  prm.num_kb = kb;
  prm.idesc = pipe::idesc(A->fmt, B->fmt, false, false, pair ? 256 : 128, 128);
  prm.split = ch.split;
  const uintptr_t bits = ca | (M > 1 ? uintptr_t(ld * es) : 0);
  prm.c_align = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;
  prm.debug_flags = o.debug_flags;
  prm.timeout_ns = timeout_ns;
  rc = op_status_word(&prm.status);
  if (rc != SWZ_OK) return rc;
  uint64_t programs = sm * sn * cl;
  if (ch.split == 1) {
    const uint64_t cap = o.num_programs ? uint64_t(o.num_programs)
                                        : uint64_t(dev.num_sms) / cl * cl;
    if (programs > cap) programs = cap;
  }
  const bool brow = B->block == SWZ_BLOCK_ROW;
  if (pair)
    return brow ? launch<true, true>(ta, tb, prm, uint32_t(programs), s)
                : launch<true, false>(ta, tb, prm, uint32_t(programs), s);
  return brow ? launch<false, true>(ta, tb, prm, uint32_t(programs), s)
              : launch<false, false>(ta, tb, prm, uint32_t(programs), s);
}
