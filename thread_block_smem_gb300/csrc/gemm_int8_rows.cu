// gemm_int8_rows.cu -- swz_gemm_int8 with few rows of A (up to 32: decoding), the
// same exact sums taken as C^T = B * A^T straight from the bytes of B.
//
// Bound: reading B once, N * K bytes.  One CTA an SM; each takes R rows of B (any
// multiple of 8, chosen so that all SMs have the same share) and their whole K, or a
// cluster of 2 to 8 CTAs shares it where N is small.  TMA brings blocks of 128 of K
// (R rows of B, and A's rows; 128-byte swizzle) into a ring that fills shared
// memory.  A warp takes 32 rows of B and one half of a block's K, widens both
// operands in registers to fp16 and multiplies them with mma.sync (B's rows are its
// M, eight rows of A its N); 2 P warps make a block (P = R / 32), and G such groups
// take the blocks in turn, so that the latency of one is under the others'.  tcgen05
// would want B's widened tile in shared memory or TMEM first, twice the bytes of
// what is read.
//   * The order of K inside a product is free as long as both operands share it: a
//     lane's 16 bytes of a row, read in one access, are its operands of four
//     MMAs.  The halves of K are the even and odd 16-byte pieces of a row, so that
//     the two rows that a quarter of a warp reads lie in different banks.
//   * An fp32 accumulator holds 1024 products exactly; every 1024 it is added to
//     an int32 total.  The warps' totals are added in shared memory, the ranks' of
//     a cluster through distributed shared memory: whole numbers, in any order.
//   * Where SMs have more than one tile, the producer runs ahead into the next one.
//   * When the kernel before in the stream is the quantiser of A, launched by the
//     same call, B's first stages are loaded while it still runs: it lets this
//     kernel start only after everything before it has completed.
//
// Measured, in a stream of them, B from memory: 4 rows of 4096 x 4096 5.9 us, 13 rows
// 6.9, 32 rows 9.2 (12.0 in gemm_int8_batch.cu's form); of 10240 x 4096 10.6, 13.4 and
// 19.2 (22.5); of 8192 x 8192 14.2, 16.5 and 22.5 (23.5).  What grows with the rows of A
// is the arithmetic: with every product but the loads left out 13 rows of 10240 x 4096
// took 10.7 us.  64 rows took 17, 32 and 43 us against 13, 25 and 26.
#include <mutex>

#include "common.h"
#include "int8.cuh"
#include "ops.h"
#include "pipe.cuh"
#include "rows.cuh"

namespace swz {
namespace i8 {

// NT: tiles of eight rows of A.  More of them, more registers a thread and fewer
// warps.
template <int NT>
struct RowsCfg {
  static constexpr int WARPS = NT <= 2 ? 20 : 14;  // that multiply, at most
  static constexpr int THREADS = (WARPS + 1) * 32;
  static constexpr int MAX_R = 16 * WARPS < 256 ? 16 * WARPS : 256;
  static constexpr int A_BYTES = NT * 8 * 128;
};

constexpr int kMaxStages = 32, kMaxGroups = 8;
constexpr int kRowsSmem = 220 * 1024;

struct RowsParams {
  void* C;
  int64_t ldc;
  const float *sa, *sb;
  int M, N, c_dtype, early_b;
  uint32_t num_kb, split, tiles;
  uint32_t R, pairs, groups, stages;  // rows of a tile, its 32s, groups of warps
  uint32_t debug_flags;
  unsigned int* status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of shared memory as 16 fp16 numbers
__device__ __forceinline__ void load_widened(uint32_t addr, uint32_t (&h)[8]) {
  uint32_t w[4];
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) widen4(w[i], h[2 * i], h[2 * i + 1]);
}

__device__ __forceinline__ uint32_t div_up_dev(uint32_t a, uint32_t b) { return (a + b - 1) / b; }

template <int NT>
__global__ void __launch_bounds__(RowsCfg<NT>::THREADS, 1)
    gemm_int8_rows_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmB, const RowsParams p) {
  using K_ = RowsCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t b_bytes = p.R * 128, stage_bytes = b_bytes + K_::A_BYTES;
  const uint32_t ring0 = ptx::smem_u32(smem);
  const uint32_t line = (p.pairs * 32 + 4);  // words from row to row of a partial tile
  int32_t* const part = reinterpret_cast<int32_t*>(smem + p.stages * stage_bytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(part + NT * 8 * line);
  const uint32_t full0 = ptx::smem_u32(bars), empty0 = full0 + 8 * p.stages;
  int* abort_flag = reinterpret_cast<int*>(bars + 2 * p.stages);
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0);  // known uniform
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t rank = p.split > 1 ? ptx::cluster_ctarank() : 0u;
  const uint32_t first_tile = blockIdx.x / p.split, tile_step = gridDim.x / p.split;
  const uint32_t kb0 = uint32_t(uint64_t(p.num_kb) * rank / p.split);
  const uint32_t kb1 = uint32_t(uint64_t(p.num_kb) * (rank + 1) / p.split);
  const uint32_t warps = 2 * p.pairs * p.groups;  // that multiply

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tmA);
    ptx::prefetch_tensormap(&tmB);
    for (uint32_t s = 0; s < p.stages; ++s) {
      ptx::mbar_init(full0 + 8 * s, 1);
      ptx::mbar_init(empty0 + 8 * s, 2 * p.pairs);
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  for (uint32_t i = threadIdx.x; i < NT * 8 * line; i += blockDim.x) part[i] = 0;
  __syncthreads();

  pipe::Ctl ctl;
  ctl.status = p.status;
  ctl.abort_flag = abort_flag;
  ctl.peer_abort = 0;
  ctl.timeout_ns = p.timeout_ns;
  bool aborted = false;

  if (warp == warps) {
    // ---------------- TMA producer ----------------
    const uint64_t pol_b = ptx::l2_policy_evict_first(), pol_a = ptx::l2_policy_evict_last();
    const bool skip = (p.debug_flags & SWZ_DEBUG_SKIP_FIRST_LOAD) != 0;
    auto load_b = [&](uint32_t tile, uint32_t kb, uint32_t stage) {
      ptx::mbar_arrive_expect_tx(full0 + 8 * stage, stage_bytes);
      if (!(skip && kb == kb0))
        ptx::tma_load_2d(ring0 + stage * stage_bytes, &tmB, full0 + 8 * stage, int32_t(kb * 128),
                         int32_t(tile * p.R), pol_b);
    };
    auto load_a = [&](uint32_t kb, uint32_t stage) {
      ptx::tma_load_2d(ring0 + stage * stage_bytes + b_bytes, &tmA, full0 + 8 * stage,
                       int32_t(kb * 128), 0, pol_a);
    };
    // the first stages need no wait for their memory
    const uint32_t first = kb1 - kb0 < p.stages ? kb1 - kb0 : p.stages;
    const bool elected = pipe::elect_one();
    if (elected && p.early_b)
      for (uint32_t i = 0; i < first; ++i) load_b(first_tile, kb0 + i, i);
    __syncwarp();
    ptx::grid_dep_wait();
    if (elected) {
      ptx::grid_dep_launch_dependents();
      for (uint32_t i = 0; i < first; ++i) {
        if (!p.early_b) load_b(first_tile, kb0 + i, i);
        load_a(kb0 + i, i);
      }
    }
    __syncwarp();
    uint32_t stage = first == p.stages ? 0 : first, phase = first == p.stages ? 0 : 1;
    uint32_t kb = kb0 + first;
    for (uint32_t tile = first_tile; tile < p.tiles && !aborted; tile += tile_step, kb = kb0) {
      for (; kb < kb1; ++kb) {
        const bool ok = pipe::wait(empty0 + 8 * stage, phase, ctl);
        if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
        if (elected) {
          load_b(tile, kb, stage);
          load_a(kb, stage);
        }
        __syncwarp();
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
    }
    if (aborted) pipe::spin_ns(50000);  // copies already issued land
    __syncwarp();
    if (p.split > 1) {  // with the others, below
      ptx::cluster_sync();
      ptx::cluster_sync();
    }
    return;
  }

  // ---------------- sums ----------------
  ptx::grid_dep_wait();
  // 32 rows of B, half of a block's K, every `groups`-th block
  const uint32_t pair = warp % p.pairs, half = warp / p.pairs % 2, group = warp / (2 * p.pairs);
  const uint32_t g = lane / 4, c = lane % 4;
  // this lane's piece of a row (the row's number mod 8 is g in every group of 8)
  const uint32_t at = g * 128 + (((2 * c + half) ^ g) << 4);
  const int es = p.c_dtype == SWZ_F32 ? 4 : 2;
  const uint32_t threads = warps * 32;
  uint32_t stage = group, phase = 0;  // of this warp's next block
  for (uint32_t tile = first_tile; tile < p.tiles; tile += tile_step) {
    float acc[2][NT][4];
    int32_t tot[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[i][t][e] = 0.0f;
          tot[i][t][e] = 0;
        }
    auto flush = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            tot[i][t][e] += __float2int_rn(acc[i][t][e]);
            acc[i][t][e] = 0.0f;
          }
    };
    uint32_t in_chunk = 0;
#pragma unroll 1
    for (uint32_t kb = kb0 + group; kb < kb1 && !aborted; kb += p.groups) {
      const bool ok = pipe::wait(full0 + 8 * stage, phase, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
      const uint32_t b = ring0 + stage * stage_bytes + pair * 4096 + at;
      const uint32_t a = ring0 + stage * stage_bytes + b_bytes + at;
      uint32_t w[2][2][8];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) load_widened(b + i * 2048 + h * 1024, w[i][h]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t x[8];
        load_widened(a + t * 1024, x);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mma_f16(acc[i][t], w[i][0][2 * j], w[i][1][2 * j], w[i][0][2 * j + 1],
                    w[i][1][2 * j + 1], x[2 * j], x[2 * j + 1]);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty0 + 8 * stage);
      stage += p.groups;
      if (stage >= p.stages) { stage -= p.stages; phase ^= 1u; }
      if (++in_chunk == 16) {  // 64 of K a block
        flush();
        in_chunk = 0;
      }
    }
    flush();
    // row m of A, row n of the tile at m * line + n words (2 line mod 32 is 8: no bank
    // conflicts)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          atomicAdd(part + (t * 8 + 2 * c + (e & 1)) * line + pair * 32 + i * 16 + g + (e & 2) * 4,
                    tot[i][t][e]);
    if (aborted) *abort_flag = 1;
    if (p.split > 1) {
      __syncwarp();
      ptx::cluster_sync();
    } else {
      asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
    }
    const bool failed = *abort_flag != 0;
    const uint32_t cols = p.R / p.split + (p.R % p.split != 0);  // this rank's columns of C
    const uint32_t part0 = ptx::smem_u32(part);
    for (uint32_t i = threadIdx.x; i < uint32_t(p.M) * cols; i += threads) {
      const uint32_t m = i / cols, n = rank * cols + i % cols;
      const int64_t col = int64_t(tile) * p.R + n;
      if (n >= p.R || col >= p.N) continue;
      int32_t sum = 0;
      if (p.split > 1) {
        const uint32_t from = part0 + (m * line + n) * 4;
        int32_t v[8];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
          v[j] = 0;
          if (j < p.split)
            asm volatile("ld.shared::cluster.s32 %0, [%1];"
                         : "=r"(v[j])
                         : "r"(ptx::map_to_rank(from, j)));
        }
        sum = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
      } else {
        sum = part[m * line + n];
        part[m * line + n] = 0;
      }
      if (!failed)
        rows::store1(static_cast<uint8_t*>(p.C) + (int64_t(m) * p.ldc + col) * es,
                     float(sum) * (p.sa[m] * p.sb[col]), p.c_dtype);
    }
    if (p.split > 1) {
      __syncwarp();
      ptx::cluster_sync();  // no CTA leaves while its partial tile is read
      return;
    }
    // the next tile's blocks follow this one's: from this warp's block after its last
    // to the first of the next tile's
    {
      const uint32_t n = kb1 - kb0;
      uint32_t own = group;  // blocks of this tile up to where `stage` stands
      own += (n > group ? div_up_dev(n - group, p.groups) : 0u) * p.groups;
      // the distance n + group - own is below the number of groups either way
      const int move = int(n + group) - int(own);
      int at_stage = int(stage) + move;
      if (at_stage >= int(p.stages)) { at_stage -= int(p.stages); phase ^= 1u; }
      if (at_stage < 0) { at_stage += int(p.stages); phase ^= 1u; }
      stage = uint32_t(at_stage);
    }
    // rows of the last group of 32 that the tile does not have, and of A beyond M
    for (uint32_t i = threadIdx.x; i < NT * 8 * line; i += threads)
      if (i / line >= uint32_t(p.M) || i % line >= p.R) part[i] = 0;
    // after a wait that ran out, too, every warp goes through all tiles (the next waits
    // return at once), so that the barriers match
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
  }
}

template <int NT>
static int launch_rows(const CUtensorMap& ta, const CUtensorMap& tb, const RowsParams& prm,
                       uint32_t ctas, cudaStream_t stream) {
  auto kern = gemm_int8_rows_kernel<NT>;
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  SWZ_CUDA_TRY(cudaGetDevice(&dev));
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      SWZ_CUDA_TRY(
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem));
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3((2 * prm.pairs * prm.groups + 1) * 32);
  cfg.dynamicSmemBytes = kRowsSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = prm.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, ta, tb, prm));
  return SWZ_OK;
}

static uint32_t div_up(uint64_t a, uint64_t b) { return uint32_t((a + b - 1) / b); }

int gemm_int8_rows(const void* A, int64_t lda, const float* sa, const void* B, int64_t ldb,
                   const float* sb, void* C, int64_t ldc, int c_dtype, int M, int N, int K,
                   int split, uint32_t debug_flags, uint64_t timeout_ns, bool early_b,
                   int num_sms, cudaStream_t stream) {
  const uint32_t kb = div_up(uint64_t(K), 128);
  const uint32_t nt = M <= 8 ? 1 : M <= 16 ? 2 : 4;
  const uint32_t max_warps = nt <= 2 ? RowsCfg<1>::WARPS : RowsCfg<4>::WARPS;
  const uint32_t max_r = nt <= 2 ? RowsCfg<1>::MAX_R : RowsCfg<4>::MAX_R;
  if (uint32_t(split) > kb) return SWZ_EUNSUPPORTED;  // an empty range of K
  // The split with the least to read for one SM: its tiles times the blocks of K times
  // the rows (a block of less than 28 takes as long as one of 28), and the cluster's
  // exchange.  Clusters of 4 and 8 leave some SMs of a group over.
  uint32_t s = 1, R = 8;
  uint64_t best = ~uint64_t(0);
  for (uint32_t t = 1; t <= 8; t *= 2) {
    if (split ? t != uint32_t(split) : (t > 1 && kb < 2 * t)) continue;
    const uint32_t clusters = uint32_t(num_sms) / t - (t >= 4 ? uint32_t(num_sms) / t / 8 : 0);
    const uint32_t per = clusters ? clusters : 1;
    const uint32_t waves = div_up(uint64_t(N), uint64_t(per) * max_r);
    const uint32_t r = (div_up(uint64_t(N), uint64_t(per) * waves) + 7) / 8 * 8;
    if (!split && t > 1 && waves > 1) continue;
    const uint64_t cost =
        uint64_t(waves) * div_up(kb, t) * (r < 28 ? 28 : r) + (t > 1 ? 250 : 0);
    if (cost < best) {
      best = cost;
      s = t;
      R = r;
    }
  }
  RowsParams p{};
  p.C = C;
  p.ldc = ldc;
  p.sa = sa;
  p.sb = sb;
  p.M = M;
  p.N = N;
  p.c_dtype = c_dtype;
  p.early_b = early_b;
  p.num_kb = kb;
  p.split = s;
  p.R = R;
  p.tiles = div_up(uint64_t(N), R);
  p.pairs = div_up(R, 32);
  p.groups = max_warps / (2 * p.pairs);
  if (p.groups > uint32_t(kMaxGroups)) p.groups = kMaxGroups;
  if (p.groups > div_up(kb, s)) p.groups = div_up(kb, s);
  const uint32_t stage = R * 128 + nt * 1024, part = nt * 8 * (p.pairs * 32 + 4) * 4;
  p.stages = (uint32_t(kRowsSmem) - 1024 - part - 2 * kMaxStages * 8 - 16) / stage;
  if (p.stages > uint32_t(kMaxStages)) p.stages = kMaxStages;
  if (p.groups > p.stages) p.groups = p.stages;
  p.debug_flags = debug_flags;
  p.timeout_ns = timeout_ns;
  CUtensorMap ta, tb;
  int rc = encode_bytes(&ta, A, uint64_t(M), uint64_t(K), uint64_t(lda), nt * 8);
  if (rc != SWZ_OK) return rc;
  rc = encode_bytes(&tb, B, uint64_t(N), uint64_t(K), uint64_t(ldb), R);
  if (rc != SWZ_OK) return rc;
  rc = op_status_word(&p.status);
  if (rc != SWZ_OK) return rc;
  if (uint64_t(p.tiles) * s > uint64_t(INT32_MAX)) return SWZ_EINVAL;
  uint32_t ctas = p.tiles * s;
  if (s == 1 && ctas > uint32_t(num_sms)) ctas = uint32_t(num_sms);
  switch (nt) {
    case 1: return launch_rows<1>(ta, tb, p, ctas, stream);
    case 2: return launch_rows<2>(ta, tb, p, ctas, stream);
    default: return launch_rows<4>(ta, tb, p, ctas, stream);
  }
}

}  // namespace i8
}  // namespace swz
