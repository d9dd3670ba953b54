// gemm_int8_batch.cu -- swz_gemm_int8 and swz_linear_int8 with a few to a few hundred
// rows of A (a decoding batch, a short prompt): the same exact sums as C^T = B * A^T,
// B read once as bytes and widened on its way to the tensor core.
//
// Bound: reading B, N * K bytes, while A's rows are few.  128 rows of B are the tensor
// core's M, the rows of A its N (a multiple of 16, up to 256).  A is there as fp16
// numbers already (written by the quantiser, or by a pass over its few bytes) and comes
// through TMA.  B's bytes come through TMA too, into a ring of blocks of 128 of K; eight
// warps read them, widen them in registers and store them to the operand's stage of 64
// of K, from which the tensor core takes them.  (B's bytes straight from global memory
// to registers, three blocks ahead, would spare shared memory a write and a read, but an
// arrival on a barrier releases what came before it, and so waits for the loads under
// way: a block then took a whole trip to memory, 0.85 us.)
//   * 11 warps: 0-7 widen, then the epilogue; 8 TMA for B, 9 for A; 10 MMA issue.  Two
//     CTAs an SM where A's stages are small.
//   * Every 1024 of K is an accumulation of its own (fp32 holds its sum exactly), in
//     columns of TMEM of its own: nothing is read back before the end, when the sums
//     are added as whole numbers.
//   * A cluster of 1 to 8 CTAs shares a tile's K; the partial tiles are added through
//     distributed shared memory.
//   * When the kernel before in the stream is the one that writes A, launched by the
//     same call, B's first blocks are loaded while it still runs: it lets this kernel
//     start only after everything before it has completed.
//
// Measured, in a stream of them, with the pass that widens A, B from memory: 64 rows
// of 4096 x 4096 14.0 us, 128 rows 14.8, 256 rows 18.6 (24 to 34 where all of B is
// widened to memory first), of 10240 x 4096 25, 32 and 49 (49 to 56), of 8192 x 8192
// 26, 33 and 49 (77 to 92).  The layer with 512 rows of 4096 x 4096 27 us (37), of 2048 x
// 2048 15 (18), of 10240 x 4096 73 (83), of 8192 x 8192 97 (96): 512 rows are the most.  A block of 128 of K takes a CTA 0.65 us, several times its
// MMAs: the way through widening, fence, MMA and release of a stage, of which two or
// three are in turn.
#include <mutex>

#include "common.h"
#include "int8.cuh"
#include "ops.h"
#include "pipe.cuh"
#include "rows.cuh"

namespace swz {
namespace i8 {

constexpr int kBatchWarps = 8, kBatchThreads = (kBatchWarps + 3) * 32;
constexpr int kBatchStages = 3;              // of the widened operands
constexpr int kBatchSlots = 8;               // of B's bytes, at most
constexpr uint32_t kBatchB = 128 * 128;      // bytes of a stage's B, and of a slot
constexpr uint32_t kHalvesOfSum = 1024 / 64;

struct BatchParams {
  const float *sa, *sb;
  uint8_t* C;
  int64_t ldc;  // elements
  int c_dtype;
  int M, N;
  uint32_t nb;      // rows of A a tile, a multiple of 16
  uint32_t tiles_m;
  uint32_t num_kb, split, stages, slots, tmem_cols, idesc;
  uint32_t debug_flags;
  unsigned int* status;
  uint64_t timeout_ns;
};

// CTAS: resident an SM
template <int CTAS>
__global__ void __launch_bounds__(kBatchThreads, CTAS)
    gemm_int8_batch_kernel(const __grid_constant__ CUtensorMap tmA,
                           const __grid_constant__ CUtensorMap tmB, const BatchParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t bars[3 * kBatchStages + 2 * kBatchSlots + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t a_bytes = p.nb * 128;  // of a stage
  // stages of the widened B, stages of A, slots of B's bytes
  const uint32_t sB = ptx::smem_u32(smem), sA = sB + p.stages * kBatchB;
  const uint32_t sQ = sA + p.stages * a_bytes;
  const uint32_t wfull0 = ptx::smem_u32(bars), xfull0 = wfull0 + 8 * kBatchStages;
  const uint32_t empty0 = xfull0 + 8 * kBatchStages, qfull0 = empty0 + 8 * kBatchStages;
  const uint32_t qempty0 = qfull0 + 8 * kBatchSlots, done_bar = qempty0 + 8 * kBatchSlots;
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0);  // known uniform
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t rank = p.split > 1 ? ptx::cluster_ctarank() : 0u;
  const uint32_t tile = blockIdx.x / p.split;
  const int m0 = int(tile % p.tiles_m) * int(p.nb);
  const int n0 = int(tile / p.tiles_m) * 128;  // (n0 + 127 may not fit 32 bits)
  const uint32_t kb0 = uint32_t(uint64_t(p.num_kb) * rank / p.split);
  const uint32_t kb1 = uint32_t(uint64_t(p.num_kb) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tmA);
    ptx::prefetch_tensormap(&tmB);
    for (uint32_t s = 0; s < uint32_t(kBatchStages); ++s) {
      ptx::mbar_init(wfull0 + 8 * s, kBatchWarps);
      ptx::mbar_init(xfull0 + 8 * s, 1);
      ptx::mbar_init(empty0 + 8 * s, 1);
    }
    for (uint32_t s = 0; s < uint32_t(kBatchSlots); ++s) {
      ptx::mbar_init(qfull0 + 8 * s, 1);
      ptx::mbar_init(qempty0 + 8 * s, kBatchWarps);
    }
    ptx::mbar_init(done_bar, 1);
    abort_word = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kBatchWarps + 2) {
    ptx::tmem_alloc<1>(ptx::smem_u32(&tmem_slot), p.tmem_cols);
    ptx::tmem_relinquish<1>();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_slot;

  pipe::Ctl ctl;
  ctl.status = p.status;
  ctl.abort_flag = &abort_word;
  ctl.peer_abort = 0;
  ctl.timeout_ns = p.timeout_ns;
  bool aborted = false;

  if (warp == kBatchWarps) {
    // ---------------- TMA producer: B's bytes ----------------
    const uint64_t pol = p.tiles_m > 1 ? ptx::l2_policy_evict_last() : ptx::l2_policy_evict_first();
    bool skip = (p.debug_flags & SWZ_DEBUG_SKIP_FIRST_LOAD) != 0;
    uint32_t slot = 0, phase = 0;
    for (uint32_t kb = kb0; kb < kb1; ++kb) {
      const bool ok = pipe::wait(qempty0 + 8 * slot, phase ^ 1u, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
      if (pipe::elect_one()) {
        ptx::mbar_arrive_expect_tx(qfull0 + 8 * slot, kBatchB);
        if (!skip)
          ptx::tma_load_2d(sQ + slot * kBatchB, &tmB, qfull0 + 8 * slot, int32_t(kb * 128), n0, pol);
      }
      __syncwarp();
      skip = false;
      if (++slot == p.slots) { slot = 0; phase ^= 1u; }
    }
    if (aborted) pipe::spin_ns(50000);  // copies already issued land
    __syncwarp();
  } else if (warp == kBatchWarps + 1) {
    // ---------------- TMA producer: A ----------------
    const uint64_t pol = ptx::l2_policy_evict_last();
    ptx::grid_dep_wait();
    if (lane == 0) ptx::grid_dep_launch_dependents();
    __syncwarp();
    uint32_t stage = 0, phase = 0;
    for (uint32_t h = 2 * kb0; h < 2 * kb1; ++h) {
      const bool ok = pipe::wait(empty0 + 8 * stage, phase ^ 1u, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
      if (pipe::elect_one()) {
        ptx::mbar_arrive_expect_tx(xfull0 + 8 * stage, a_bytes);
        ptx::tma_load_3d(sA + stage * a_bytes, &tmA, xfull0 + 8 * stage, int32_t(h * 64), m0, 0,
                         pol);
      }
      __syncwarp();
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
    // every stage released: nothing is in flight towards this CTA
    for (uint32_t i = 0; i < p.stages && !aborted; ++i) {
      const bool ok = pipe::wait(empty0 + 8 * stage, phase ^ 1u, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) aborted = true;
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
    if (aborted) pipe::spin_ns(50000);  // copies already issued land
    __syncwarp();
  } else if (warp == kBatchWarps + 2) {
    // ---------------- MMA issuer ----------------
    uint32_t stage = 0, phase = 0;
    bool issued = false;
    const uint64_t bdesc0 = pipe::sdesc128(sB, 16, 1024), adesc0 = pipe::sdesc128(sA, 16, 1024);
    for (uint32_t h = 2 * kb0; h < 2 * kb1; ++h) {
      const bool ok = pipe::wait(xfull0 + 8 * stage, phase, ctl) &&
                      pipe::wait(wfull0 + 8 * stage, phase, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
      ptx::tc_fence_after();
      const uint32_t sum = (h - 2 * kb0) / kHalvesOfSum, in_sum = (h - 2 * kb0) % kHalvesOfSum;
      if (pipe::elect_one()) {
#pragma unroll
        for (uint32_t kk = 0; kk < 4; ++kk)
          ptx::mma<1, 0>(tmem_base + sum * p.nb, bdesc0 + ((stage * kBatchB) >> 4) + kk * 2,
                         adesc0 + ((stage * a_bytes) >> 4) + kk * 2, p.idesc, (in_sum | kk) != 0);
        ptx::mma_commit(empty0 + 8 * stage);
        if (h + 1 == 2 * kb1) ptx::mma_commit(done_bar);
      }
      __syncwarp();
      issued = true;
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
    if (aborted && issued) {
      // drain: wait (bounded) until every MMA issued so far has completed
      if (pipe::elect_one()) ptx::mma_commit(done_bar);
      const uint64_t t0 = ptx::global_timer_ns();
      while (!pipe::try_wait(done_bar, 0) && ptx::global_timer_ns() - t0 < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else {
    // ---------------- widening ----------------
    // 16 bytes of 64 of K of a row a thread: rows r and r + 64, piece c of four.  Eight
    // lanes that access shared memory together have two rows four apart, whose pieces lie
    // in different halves of the (swizzled) line of B's bytes; of the widened line, where
    // they have the same even or odd pieces, one of the two rows takes the odd ones first.
    const uint32_t r = warp * 8 + ((lane >> 3) & 3u) + (lane & 4u), c = lane & 3u;
    const uint32_t swap = (lane >> 2) & 1u, x = r & 7u;
    const uint32_t from0 = sQ + r * 128 + ((c ^ x) << 4), from1 = sQ + r * 128 + (((4 + c) ^ x) << 4);
    uint8_t* const to0 = smem + r * 128 + (((2 * c + swap) ^ x) << 4);
    uint8_t* const to1 = smem + r * 128 + (((2 * c + (swap ^ 1u)) ^ x) << 4);
    uint32_t slot = 0, q_phase = 0, stage = 0, phase = 0;
    for (uint32_t kb = kb0; kb < kb1 && !aborted; ++kb) {
      if (!__all_sync(0xFFFFFFFFu, pipe::wait(qfull0 + 8 * slot, q_phase, ctl))) {
        aborted = true;
        break;
      }
      uint32_t v[2][2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[h][i][0]), "=r"(v[h][i][1]), "=r"(v[h][i][2]), "=r"(v[h][i][3])
                       : "r"((h ? from1 : from0) + slot * kBatchB + i * 8192)
                       : "memory");
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!__all_sync(0xFFFFFFFFu, pipe::wait(empty0 + 8 * stage, phase ^ 1u, ctl))) {
          aborted = true;
          break;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) widen4(v[h][i][e], w[2 * e], w[2 * e + 1]);
          const uint4 lo = make_uint4(w[0], w[1], w[2], w[3]);
          const uint4 hi = make_uint4(w[4], w[5], w[6], w[7]);
          *reinterpret_cast<uint4*>(to0 + stage * kBatchB + i * 8192) = swap ? hi : lo;
          *reinterpret_cast<uint4*>(to1 + stage * kBatchB + i * 8192) = swap ? lo : hi;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(wfull0 + 8 * stage);
          if (h == 0) ptx::mbar_arrive(qempty0 + 8 * slot);  // in registers since
        }
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
      if (++slot == p.slots) { slot = 0; q_phase ^= 1u; }
    }
    const bool ok = !aborted && pipe::wait(done_bar, 0, ctl);
    if (!__all_sync(0xFFFFFFFFu, ok)) aborted = true;
    ptx::tc_fence_after();
    ptx::grid_dep_wait();
  }

  // ---------------- epilogue ----------------
  // warp w: rows 32 (w mod 4) .. of B's tile, every second 16 rows of A
  const uint32_t q = warp & 3u;
  const uint32_t sums = (2 * (kb1 - kb0) + kHalvesOfSum - 1) / kHalvesOfSum;
  const int es = p.c_dtype == SWZ_F32 ? 4 : 2;
  int32_t* const part = reinterpret_cast<int32_t*>(smem);  // nb rows of 128, over the stages and
  // slots (every MMA has completed, and so every load that it waited for)
  if (warp < kBatchWarps && !aborted) {
    const int64_t n = n0 + int64_t(q * 32 + lane);
    const float sb = n < p.N ? p.sb[n] : 0.0f;
    for (uint32_t m = warp / 4 * 16; m < p.nb; m += 32) {
      if (m0 + int(m) >= p.M) break;
      int32_t total[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) total[j] = 0;
      for (uint32_t i = 0; i < sums; ++i) {
        uint32_t v[16];
        pipe::tmem_ld16(tmem_base + ((q * 32u) << 16) + i * p.nb + m, v);
        pipe::tmem_ld_wait16(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) total[j] += __float2int_rn(__uint_as_float(v[j]));
      }
      if (p.split > 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(m + j) * 128 + q * 32 + lane] = total[j];
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int64_t row = m0 + int64_t(m) + j;
          if (row < p.M && n < p.N)
            rows::store1(p.C + (row * p.ldc + n) * es, float(total[j]) * (p.sa[row] * sb),
                         p.c_dtype);
        }
      }
    }
  }
  if (p.split > 1) {
    __syncwarp();
    ptx::cluster_sync();
    if (warp < kBatchWarps && !aborted) {
      // rank r takes every split-th row of A, a warp a row, a lane four columns
      const int64_t n = n0 + int64_t(lane) * 4;
      float sb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sb[e] = n + e < p.N ? p.sb[n + e] : 0.0f;
      const uint32_t part0 = ptx::smem_u32(part);
      for (uint32_t m = rank + p.split * warp; m < p.nb; m += p.split * kBatchWarps) {
        const int64_t at = m0 + int64_t(m);
        if (at >= p.M) break;
        int32_t v[8][4];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
          v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0;
          if (j < p.split)
            asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[j][0]), "=r"(v[j][1]), "=r"(v[j][2]), "=r"(v[j][3])
                         : "r"(ptx::map_to_rank(part0 + (m * 128 + lane * 4) * 4, j)));
        }
        const float sa = p.sa[at];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int32_t s = 0;
#pragma unroll
          for (uint32_t j = 0; j < 8; ++j) s += v[j][e];
          if (n + e < p.N)
            rows::store1(p.C + (at * p.ldc + n + e) * es, float(s) * (sa * sb[e]), p.c_dtype);
        }
      }
    }
    __syncwarp();
    ptx::cluster_sync();  // no CTA leaves while its partial tile is read
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kBatchWarps + 2) ptx::tmem_dealloc<1>(tmem_base, p.tmem_cols);
}

template <int CTAS>
static int launch_batch(const CUtensorMap& ta, const CUtensorMap& tb, const BatchParams& prm, uint32_t ctas,
                        uint32_t smem, cudaStream_t stream) {
  auto kern = gemm_int8_batch_kernel<CTAS>;
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  SWZ_CUDA_TRY(cudaGetDevice(&dev));
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      SWZ_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        224 * 1024 / CTAS));
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kBatchThreads);
  cfg.dynamicSmemBytes = smem;
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

// How M x N x K is cut; split 0 where K is too long for the tensor memory.
BatchPlan batch_plan(int M, int N, int K, int split, int num_sms) {
  BatchPlan b{};
  b.tiles_m = div_up(uint64_t(M), 256);
  b.nb = (div_up(uint64_t(M), b.tiles_m) + 15) / 16 * 16;
  b.ctas_per_sm = b.nb <= 64 ? 2 : 1;
  const uint32_t stage = kBatchB + b.nb * 128, room = 224u * 1024 / b.ctas_per_sm - 2048;
  b.stages = b.ctas_per_sm == 2 ? 2 : kBatchStages;
  b.slots = (room - b.stages * stage) / kBatchB;
  if (b.slots > uint32_t(kBatchSlots)) b.slots = kBatchSlots;
  const uint64_t tiles = uint64_t(b.tiles_m) * div_up(uint64_t(N), 128);
  const uint32_t kb = div_up(uint64_t(K), 128), most = 512 / b.ctas_per_sm;
  auto columns = [&](uint32_t s) { return div_up(2 * div_up(kb, s), kHalvesOfSum) * b.nb; };
  uint32_t s = split ? uint32_t(split) : 1;
  if (!split)
    // As many CTAs as stay resident, each with a block of K at least.  Clusters of 4 and 8
    // leave some SMs of a group over: 16 clusters of 8 do not fit one CTA an SM (400 rows of
    // 1024 x 8192, 16 tiles: 31.5 us by eight, 24.3 by four).
    while (s < 8 && (columns(s) > most ||
                     (tiles * s * 2 <= uint64_t(num_sms) * b.ctas_per_sm * (s == 4 ? 6 : s == 2 ? 7 : 8) / 8 &&
                      kb >= 2 * s)))
      s *= 2;
  if (s > kb || columns(s) > most) return b;
  b.split = s;
  b.tmem_cols = 32;
  while (b.tmem_cols < columns(s)) b.tmem_cols *= 2;
  b.tiles = tiles;
  return b;
}

int gemm_int8_batch(const void* a16, int64_t ld, const float* sa, const void* B, int64_t ldb,
                    const float* sb, void* C, int64_t ldc, int c_dtype, int M, int N, int K,
                    const BatchPlan& b, uint32_t debug_flags, uint64_t timeout_ns,
                    cudaStream_t stream) {
  if (b.tiles * b.split > uint64_t(INT32_MAX)) return SWZ_EINVAL;
  CUtensorMap ta, tb;
  int rc = encode_half(&ta, a16, 1, uint64_t(M), uint64_t(K), uint64_t(ld),
                       uint64_t(M) * uint64_t(ld), 64, b.nb);
  if (rc != SWZ_OK) return rc;
  rc = encode_bytes(&tb, B, uint64_t(N), uint64_t(K), uint64_t(ldb), 128);
  if (rc != SWZ_OK) return rc;
  BatchParams p{};
  p.sa = sa;
  p.sb = sb;
  p.C = static_cast<uint8_t*>(C);
  p.ldc = ldc;
  p.c_dtype = c_dtype;
  p.M = M;
  p.N = N;
  p.nb = b.nb;
  p.tiles_m = b.tiles_m;
  p.num_kb = div_up(uint64_t(K), 128);
  p.split = b.split;
  p.stages = b.stages;
  p.slots = b.slots;
  p.tmem_cols = b.tmem_cols;
  p.idesc = pipe::idesc(0, 0, false, false, 128, int(b.nb));
  p.debug_flags = debug_flags;
  p.timeout_ns = timeout_ns;
  rc = op_status_word(&p.status);
  if (rc != SWZ_OK) return rc;
  const uint32_t ctas = uint32_t(b.tiles * b.split);
  const uint32_t smem = 1024 + b.stages * (kBatchB + b.nb * 128) + b.slots * kBatchB;
  return b.ctas_per_sm == 2 ? launch_batch<2>(ta, tb, p, ctas, smem, stream)
                            : launch_batch<1>(ta, tb, p, ctas, smem, stream);
}

}  // namespace i8
}  // namespace swz
