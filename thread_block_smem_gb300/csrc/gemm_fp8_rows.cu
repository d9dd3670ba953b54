// gemm_fp8_rows.cu -- swz_gemm_fp8 with few rows of A (up to 32: decoding):
// the same sums, taken as C^T = B * A^T.
//
// Bound: reading B once, N * K bytes.  A 128-row tile of A would be mostly
// padding and its 128 x 128 accumulators most of the work, so the operands
// change places: 128 rows of B are the tensor core's M, the rows of A its N
// (16 or 32).  A block of K is then 16 KB of B through TMA, one small MMA
// group, and 16 or 32 columns of TMEM to scale and add; the stages of two CTAs keep
// up to 160 KB of B (128 with 32 rows) in flight on an SM.
//   * 7 warps: 0-3 the sums (TMEM lanes 32 w .., one row of B a thread), 4 TMA
//     producer, 5 MMA issue, 6 scales.
//   * A cluster of 1 to 8 CTAs shares a tile's K; the partial tiles are added
//     through distributed shared memory in rank order, each rank storing its
//     share of the rows of C.  With the remote reads of a row after another's
//     16 rows of 10240 x 4096 took 12.6 us, with all of them in flight 10.9.
//   * When the kernel before in the stream is the quantiser of A, launched by
//     the same call, B's first stages are loaded while it still runs: it lets
//     this kernel start only after everything before it has completed.
//
// Measured, in a stream of them, B from memory: one row of 4096 x 4096 6.2 us
// (2.7 TB/s), 10240 x 4096 10.5 (4.0), 8192 x 8192 13.8 (4.9), 28672 x 4096 22.7
// (5.2).  About 2.8 us are start, first load and the last block's way out;
// what follows them runs at the copy bandwidth.
#include <mutex>
#include <type_traits>

#include "common.h"
#include "f8.cuh"
#include "ops.h"
#include "pipe.cuh"

namespace swz {
namespace gemm8 {

constexpr int kRowsThreads = 7 * 32;
constexpr int kRowsSlots = 3, kSlotKb = 4;  // ring of scales: slots of four blocks

template <int BN>
struct RowsCfg {
  static constexpr int B_BYTES = 128 * 128, A_BYTES = BN * 128;
  static constexpr int STAGE = B_BYTES + A_BYTES;
  static constexpr int STAGES = BN == 16 ? 5 : 4;  // two CTAs an SM
  static constexpr int NBUF = 4, TMEM_COLS = 4 * BN;
  static constexpr int SLOT = 128 + BN;  // scales of a block: B's rows, then A's
  static constexpr int BARS = 2 * STAGES + 2 * NBUF + 2 * kRowsSlots + 1;
  static constexpr int SMEM =
      1024 + STAGES * STAGE + kRowsSlots * kSlotKb * SLOT * 4 + BARS * 8 + 16;
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs an SM");
  static_assert(STAGES * STAGE >= 128 * BN * 4, "a partial tile fits the ring");
};

struct RowsParams {
  void* C;
  int64_t ldc;
  const float *sa, *sb;
  int64_t ldsa, ldsb;
  int M, N, c_dtype, b_square, early_b;
  int c_quads;  // four results of a row are one aligned store
  uint32_t num_kb, idesc, split;
  uint32_t debug_flags;
  unsigned int* status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ uint32_t pack2_out(float a, float b, int dtype) {
  if (dtype == SWZ_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store_out(void* C, int64_t at, float v, int dtype) {
  if (dtype == SWZ_F32) static_cast<float*>(C)[at] = v;
  else if (dtype == SWZ_BF16) static_cast<__nv_bfloat16*>(C)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(C)[at] = __float2half_rn(v);
}

template <int BN>
__global__ void __launch_bounds__(kRowsThreads, 2)
    gemm_fp8_rows_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB, const RowsParams p) {
  using K_ = RowsCfg<BN>;
  constexpr uint32_t STAGES = K_::STAGES, NBUF = K_::NBUF, SLOTS = kRowsSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sB = ptx::smem_u32(smem);
  const uint32_t sA = sB + STAGES * K_::B_BYTES;
  const uint32_t ring0 = sB + STAGES * K_::STAGE;
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(smem + STAGES * K_::STAGE +
                                  SLOTS * kSlotKb * K_::SLOT * 4);
  const uint32_t full0 = ptx::smem_u32(bars), empty0 = full0 + 8 * STAGES;
  const uint32_t tfull0 = empty0 + 8 * STAGES, tempty0 = tfull0 + 8 * NBUF;
  const uint32_t sfull0 = tempty0 + 8 * NBUF, sempty0 = sfull0 + 8 * SLOTS;
  const uint32_t drain_bar = sempty0 + 8 * SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + K_::BARS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0);  // known uniform
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t rank = p.split > 1 ? ptx::cluster_ctarank() : 0u;

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tmA);
    ptx::prefetch_tensormap(&tmB);
    for (uint32_t s = 0; s < STAGES; ++s) {
      ptx::mbar_init(full0 + 8 * s, 1);
      ptx::mbar_init(empty0 + 8 * s, 1);
    }
    for (uint32_t a = 0; a < NBUF; ++a) {
      ptx::mbar_init(tfull0 + 8 * a, 1);
      ptx::mbar_init(tempty0 + 8 * a, 4);
    }
    for (uint32_t i = 0; i < SLOTS; ++i) {
      ptx::mbar_init(sfull0 + 8 * i, 32);
      ptx::mbar_init(sempty0 + 8 * i, 4);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 5) {
    ptx::tmem_alloc<1>(ptx::smem_u32(tmem_slot), K_::TMEM_COLS);
    ptx::tmem_relinquish<1>();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pipe::Ctl ctl;
  ctl.status = p.status;
  ctl.abort_flag = abort_flag;
  ctl.peer_abort = 0;
  ctl.timeout_ns = p.timeout_ns;

  const uint32_t tile = blockIdx.x / p.split;
  const int64_t n0 = int64_t(tile) * 128;
  const uint32_t kb0 = uint32_t(uint64_t(p.num_kb) * rank / p.split);
  const uint32_t kb1 = uint32_t(uint64_t(p.num_kb) * (rank + 1) / p.split);
  bool aborted = false;
  float acc[BN];

  if (warp == 4) {
    // ---------------- TMA producer ----------------
    const uint64_t pol_b = ptx::l2_policy_evict_first(), pol_a = ptx::l2_policy_evict_last();
    const bool skip = (p.debug_flags & SWZ_DEBUG_SKIP_FIRST_LOAD) != 0;
    const uint32_t n = kb1 - kb0, first = n < STAGES ? n : STAGES;
    auto load_b = [&](uint32_t i, uint32_t stage) {
      ptx::mbar_arrive_expect_tx(full0 + 8 * stage, K_::STAGE);
      if (!(skip && i == 0))
        ptx::tma_load_2d(sB + stage * K_::B_BYTES, &tmB, full0 + 8 * stage,
                         int32_t((kb0 + i) * 128), int32_t(n0), pol_b);
    };
    auto load_a = [&](uint32_t i, uint32_t stage) {
      ptx::tma_load_2d(sA + stage * K_::A_BYTES, &tmA, full0 + 8 * stage,
                       int32_t((kb0 + i) * 128), 0, pol_a);
    };
    if (!p.early_b) ptx::grid_dep_wait();
    if (pipe::elect_one())
      for (uint32_t i = 0; i < first; ++i) load_b(i, i);
    __syncwarp();
    if (p.early_b) ptx::grid_dep_wait();
    if (pipe::elect_one()) {
      ptx::grid_dep_launch_dependents();
      for (uint32_t i = 0; i < first; ++i) load_a(i, i);
    }
    __syncwarp();
    uint32_t stage = 0, phase = 0;
    for (uint32_t i = first; i < n; ++i) {
      const bool ok = pipe::wait(empty0 + 8 * stage, phase, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
      if (pipe::elect_one()) {
        load_b(i, stage);
        load_a(i, stage);
      }
      __syncwarp();
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    }
    // the stages in use released: no commit is in flight towards this CTA
    for (uint32_t i = 0; i < first && !aborted; ++i) {
      const bool ok = pipe::wait(empty0 + 8 * stage, phase, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) aborted = true;
      if (++stage == first) { stage = 0; phase ^= 1u; }
    }
    if (aborted) pipe::spin_ns(50000);  // copies already issued land
    __syncwarp();
  } else if (warp == 5) {
    // ---------------- MMA issuer ----------------
    // what the kernel before takes does not count against this one's bound
    ptx::grid_dep_wait();
    uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
    bool issued = false;
    const uint64_t bdesc = pipe::sdesc128(sB, 16, 1024), adesc = pipe::sdesc128(sA, 16, 1024);
    for (uint32_t kb = kb0; kb < kb1; ++kb) {
      const bool ok = pipe::wait(full0 + 8 * stage, phase, ctl) &&
                      pipe::wait(tempty0 + 8 * buf, buf_phase ^ 1u, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
      ptx::tc_fence_after();
      const uint64_t b = bdesc + uint64_t(stage * uint32_t(K_::B_BYTES >> 4));
      const uint64_t a = adesc + uint64_t(stage * uint32_t(K_::A_BYTES >> 4));
      const uint32_t d = tmem_base + buf * BN;
      if (pipe::elect_one()) {
#pragma unroll
        for (uint32_t kk = 0; kk < 4; ++kk)
          pipe::mma_f8<1>(d, b + kk * 2, a + kk * 2, p.idesc, kk != 0);
        ptx::mma_commit(tfull0 + 8 * buf);
        ptx::mma_commit(empty0 + 8 * stage);
      }
      __syncwarp();
      issued = true;
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
    }
    if (aborted && issued) {
      if (pipe::elect_one()) ptx::mma_commit(drain_bar);
      const uint64_t t0 = ptx::global_timer_ns();
      while (!pipe::try_wait(drain_bar, 0) && ptx::global_timer_ns() - t0 < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else if (warp == 6) {
    // ---------------- scales ----------------
    ptx::grid_dep_wait();
    uint32_t slot = 0, phase = 0;
    for (uint32_t kb = kb0; kb < kb1; kb += kSlotKb) {
      const bool ok = pipe::wait(sempty0 + 8 * slot, phase ^ 1u, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
#pragma unroll 1
      for (uint32_t i = 0; i < uint32_t(kSlotKb) && kb + i < kb1; ++i) {
        const uint32_t dst = ring0 + (slot * kSlotKb + i) * (K_::SLOT * 4) + lane * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = n0 + lane + j * 32;
          const float* s = p.b_square ? p.sb + int64_t(tile) * p.ldsb + kb + i
                                      : p.sb + int64_t(kb + i) * p.ldsb + n;
          pipe::copy4(dst + j * 128, s, n < p.N, p.sb);
        }
#pragma unroll
        for (int j = 0; j < (BN + 31) / 32; ++j) {
          const int m = int(lane) + j * 32;
          if (m < BN)
            pipe::copy4(dst + (128 + j * 32) * 4, p.sa + int64_t(kb + i) * p.ldsa + m, m < p.M,
                        p.sa);
        }
      }
      pipe::copies_arrive(sfull0 + 8 * slot);
      if (++slot == SLOTS) { slot = 0; phase ^= 1u; }
    }
    pipe::copies_wait();
    __syncwarp();
  } else {
    // ---------------- sums: one row of B a thread, a row of A a register ----------------
    ptx::grid_dep_wait();
    uint32_t buf = 0, buf_phase = 0, slot = 0, slot_phase = 0;
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[j] = 0.f;
    const uint32_t taddr0 = tmem_base + ((warp * 32u) << 16);
#pragma unroll 1
    for (uint32_t kb = kb0; kb < kb1 && !aborted; kb += kSlotKb) {
      // one vote for four blocks: after a wait that ran out the next ones
      // return at once (the abort flag), and what is summed is not used
      const bool ok = pipe::wait(sfull0 + 8 * slot, slot_phase, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok && *abort_flag == 0)) { aborted = true; break; }
      uint32_t sc = ring0 + slot * (kSlotKb * K_::SLOT * 4);
      const uint32_t sc_end = sc + min(kb1 - kb, uint32_t(kSlotKb)) * (K_::SLOT * 4);
#pragma unroll 1
      for (; sc != sc_end; sc += K_::SLOT * 4) {
        const float s = pipe::ld_shared(sc + (warp * 32 + lane) * 4);
        pipe::wait(tfull0 + 8 * buf, buf_phase, ctl);
        __syncwarp();
        ptx::tc_fence_after();
        uint32_t r[BN / 16][16];
#pragma unroll
        for (int c = 0; c < BN / 16; ++c) pipe::tmem_ld16(taddr0 + buf * BN + c * 16, r[c]);
#pragma unroll
        for (int c = 0; c < BN / 16; ++c) pipe::tmem_ld_wait16(r[c]);
        // in registers: the tensor core may have the buffer
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(tempty0 + 8 * buf);
#pragma unroll
        for (int j = 0; j < BN / 4; ++j) {
          float a[4];
          pipe::ld_shared4(sc + (128 + 4 * j) * 4, a);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[4 * j + i] =
                fmaf(__uint_as_float(r[j / 4][(j % 4) * 4 + i]), a[i] * s, acc[4 * j + i]);
        }
        if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(sempty0 + 8 * slot);
      if (++slot == SLOTS) { slot = 0; slot_phase ^= 1u; }
    }
    const uint32_t r = warp * 32 + lane;
    if (!aborted) {
      if (p.split == 1) {
#pragma unroll
        for (int j = 0; j < BN; ++j)
          if (j < p.M && n0 + r < p.N)
            store_out(p.C, int64_t(j) * p.ldc + n0 + r, acc[j], p.c_dtype);
      } else {
        // partial tile over the ring (every load has been consumed): row j of
        // C, 128 columns
#pragma unroll
        for (int j = 0; j < BN; ++j)
          if (j < p.M) reinterpret_cast<float*>(smem)[j * 128 + r] = acc[j];
      }
    }
  }

  if (p.split > 1) {
    __syncwarp();
    ptx::cluster_sync();
    if (warp < 4 && !aborted) {
      // Rank r of S stores the rows r, r + S, .. of C: a warp a row, a lane four
      // columns, and all of a warp's remote reads (about 1 us each) in flight
      // at once.
      auto reduce = [&](auto ranks) {
        constexpr uint32_t S = decltype(ranks)::value;
        constexpr uint32_t RW = BN / (4 * S) > 0 ? BN / (4 * S) : 1;  // rows of a warp
        float f[RW][S][4];
#pragma unroll
        for (uint32_t k = 0; k < RW; ++k) {
          const uint32_t j = (rank + S * (warp + 4 * k)) % BN;  // stored only where below M
#pragma unroll
          for (uint32_t i = 0; i < S; ++i)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(f[k][i][0]), "=f"(f[k][i][1]), "=f"(f[k][i][2]), "=f"(f[k][i][3])
                         : "r"(ptx::map_to_rank(sB + (j * 128 + lane * 4) * 4, i))
                         : "memory");
        }
        const int64_t n = n0 + lane * 4;
#pragma unroll
        for (uint32_t k = 0; k < RW; ++k) {
          const uint32_t j = rank + S * (warp + 4 * k);
          if (int(j) >= p.M) continue;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = f[k][0][e];
#pragma unroll
            for (uint32_t i = 1; i < S; ++i) v[e] += f[k][i][e];
          }
          const int64_t at = int64_t(j) * p.ldc + n;
          if (p.c_quads && n + 4 <= p.N) {
            if (p.c_dtype == SWZ_F32)
              *reinterpret_cast<float4*>(static_cast<float*>(p.C) + at) =
                  make_float4(v[0], v[1], v[2], v[3]);
            else
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + at) =
                  make_uint2(pack2_out(v[0], v[1], p.c_dtype), pack2_out(v[2], v[3], p.c_dtype));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < p.N) store_out(p.C, at + e, v[e], p.c_dtype);
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
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 5) ptx::tmem_dealloc<1>(tmem_base, K_::TMEM_COLS);
}

template <int BN>
static int launch_rows(const CUtensorMap& ta, const CUtensorMap& tb, const RowsParams& prm,
                       uint32_t ctas, cudaStream_t stream) {
  using K_ = RowsCfg<BN>;
  auto kern = gemm_fp8_rows_kernel<BN>;
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  SWZ_CUDA_TRY(cudaGetDevice(&dev));
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      SWZ_CUDA_TRY(
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, K_::SMEM));
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = K_::SMEM;
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

}  // namespace gemm8

// Arguments checked by the caller; 1 <= M <= kFewRows.
int gemm_fp8_rows(const swz_fp8_matrix& A, const swz_fp8_matrix& B, void* C, int64_t ldc,
                  int c_dtype, int M, int N, int K, int split, uint32_t debug_flags,
                  uint64_t timeout_ns, bool early_b, int num_sms, cudaStream_t stream) {
  using namespace gemm8;
  const int bn = M <= 16 ? 16 : 32;
  CUtensorMap ta, tb;
  int rc = encode_bytes(&ta, A.data, uint64_t(M), uint64_t(K), uint64_t(A.ld), uint32_t(bn));
  if (rc != SWZ_OK) return rc;
  rc = encode_bytes(&tb, B.data, uint64_t(N), uint64_t(K), uint64_t(B.ld), 128);
  if (rc != SWZ_OK) return rc;
  RowsParams p{};
  p.C = C;
  p.ldc = ldc;
  p.sa = A.scales;
  p.sb = B.scales;
  p.ldsa = A.ld_scales;
  p.ldsb = B.ld_scales;
  p.M = M;
  p.N = N;
  p.c_dtype = c_dtype;
  const uintptr_t es = c_dtype == SWZ_F32 ? 4 : 2;
  p.c_quads = ((reinterpret_cast<uintptr_t>(C) | (M > 1 ? uintptr_t(ldc) * es : 0)) % (4 * es)) == 0;
  p.b_square = B.block == SWZ_BLOCK_SQUARE;
  p.early_b = early_b;
  p.num_kb = uint32_t((int64_t(K) + 127) / 128);
  p.idesc = pipe::idesc(B.fmt, A.fmt, false, false, 128, bn);
  p.debug_flags = debug_flags;
  p.timeout_ns = timeout_ns;
  rc = op_status_word(&p.status);
  if (rc != SWZ_OK) return rc;
  // K is shared by as many CTAs as stay resident (two an SM), each with four
  // blocks or more.  One row of 10240 x 4096, by CTAs of a tile (1, 2, 4, 8):
  // 12.3, 10.5, 13.7, 15.8 us; of 1024 x 8192: 19.4, 11.4, 7.2, 5.6.
  const uint64_t tiles = (uint64_t(N) + 127) / 128;
  uint32_t s = uint32_t(split);
  if (s == 0)
    for (s = 1; s < 8 && tiles * s * 2 <= uint64_t(num_sms) * 2 && p.num_kb >= 8 * s;) s *= 2;
  p.split = s;
  if (tiles * s > uint64_t(INT32_MAX)) return SWZ_EINVAL;
  const uint32_t ctas = uint32_t(tiles * s);
  return bn == 16 ? launch_rows<16>(ta, tb, p, ctas, stream)
                  : launch_rows<32>(ta, tb, p, ctas, stream);
}
}  // namespace swz
