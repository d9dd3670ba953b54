// newton_schulz.cu -- the orthogonalised update: X = G / (|G|_F + eps), then
// `steps` times
//     A = X X^T,  B = b A + c A^2,  X = a X + B X          (m <= n)
//     A = X^T X,  B = b A + c A^2,  X = a X + X B          (m >  n)
// for a batch of m x n matrices, so the square products are on the short side.
//
// Mathematics and precision: the products run on the tensor cores with fp16
// operands and fp32 sums.  What is rounded to fp16 is scaled by a power of two
// first: singular values stay below a bound that the host steps through the
// polynomial, which bounds every entry of X, A and B; the first X is G itself
// times a power of two, the exact 1 / (|G| + eps) goes into the epilogues.
// bf16 operands (8 times coarser) left the result 1 % off on normal matrices,
// fp16 ones 0.1 %.  Directions with small singular values come out of the a X
// term alone, growing by a at each step, and a rounding of X to fp16 would grow
// with them: so the a X term takes X in fp32 (G itself in the first step) in
// all steps but the last two, whose roundings no longer grow by more than a^2
// (a matrix of rank 16 plus 1 % noise: 0.03 % off instead of 4 %).  In the last
// two steps it takes the fp16 X that the products take: an error that both
// terms share is contracted by the polynomial near 1, one of them alone is not.
// Near the end A and B are nearly diagonal, so most of what B's rounding loses
// is on its diagonal.  That is kept in fp32 and given back through the a X term,
// X' = (a + lost) X + B X: 33 x 2000 0.12 % off instead of 0.20, 1024 x 1024 0.07
// instead of 0.10.
//
// Bound: the tensor cores (three products a step).  A and A^2 are symmetric:
// only tiles on and above the diagonal are computed, the epilogue writes both
// halves, which saves a third of the work of a square matrix.
//
// Kernel: as the library's GEMM -- one CTA (128 x 128 or 128 x 64) or a CTA pair
// (256 x 256) per tile, persistent; warp 8 TMA producer, warp 9 MMA issuer, warps 0-7
// epilogue (TMEM lanes 32 (w mod 4) .., columns half w / 4), two tiles of TMEM
// in turn so that an epilogue overlaps the next tile's products.  X as a
// K x N operand is read N-major from shared memory, X^T X takes both operands
// so, and nothing is ever transposed in memory.
//
// Measured, fp32 G, five steps: 4096 x 4096 945-970 us in short runs (1.42 PFLOP/s of
// the products computed, 0.75 of the measured bf16 peak) and 1060 in a stream of
// seconds, at 1.75 GHz under the power cap; 2048 x 2048 238, 1024 x 1024 113.  The pair
// kernel spills 48 bytes a thread, the 128-wide one 8, the 64-wide one nothing.
// Below 2048 it is 17 launches of 5 to 10 us that depend on one another: a
// launch's first load, its last tile's epilogue and the next one's start are not
// hidden by anything.
#include <math.h>

#include <mutex>
#include <type_traits>

#include "common.h"
#include "f8.cuh"
#include "newton_schulz.cuh"
#include "ops.h"
#include "pipe.cuh"
#include "tile_order.cuh"

namespace swz {
namespace ns {

constexpr int BM = 128;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarps + 2) * 32;

template <int BN, bool PAIR>
struct Cfg {
  static constexpr int CG = PAIR ? 2 : 1;
  static constexpr int KA = PAIR ? 1 : 2;              // 64-element atoms of K in a stage
  static constexpr int BN_LOCAL = PAIR ? BN / 2 : BN;  // columns this CTA loads
  static constexpr int A_BYTES = 128 * 128 * KA, B_BYTES = BN_LOCAL * 128 * KA;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int HALVES = BN == 64 ? 1 : 2;      // columns of a tile, by epilogue warps
  static constexpr int STAGES = 192 * 1024 / STAGE_BYTES;
  static constexpr int BARS = 2 * STAGES + 5;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + BARS * 8 + 16;
};

// What an epilogue makes of a tile's sums.
enum Mode : int {
  kGram = 0,    // A = f * acc, both halves
  kPoly = 1,    // B = u * A + f * acc, both halves
  kUpdate = 2,  // X' = factor * X + f * acc
};

// X as the a X term reads it
enum Source : int { kFromG = 0, kFromF32 = 1, kFromF16 = 2 };

struct Params {
  int mode;
  uint32_t a_mn, b_mn;          // operands given K x rows
  uint32_t tiles_m, tiles_n;    // scheduler grid of one matrix
  uint32_t per_matrix, units;   // tiles of one matrix (upper triangle when symmetric), of all
  uint32_t num_kb;              // stages of K
  uint32_t idesc;
  int M, N;                     // of the result
  // results and what they are made of, fp16 with rows ld elements apart (a
  // multiple of 16) unless said otherwise
  __half* out;
  int64_t ld_out, batch_out;
  const __half* in;             // kPoly: A; kUpdate from fp16: X
  int64_t ld_in, batch_in;
  float f, u;                   // factors (see Mode)
  const Scale* scale;           // of the batch
  int first;                    // the first step's X
  int source;                   // kUpdate
  float a;                      // kPoly, for the factors
  float out_scale;              // kUpdate: X' times out_scale goes to `out`
  // a plus what B's diagonal lost in rounding (kPoly: written; kUpdate: times X,
  // by its rows or its columns)
  float* factor;
  int64_t batch_factor;
  float lost_scale;             // kPoly: from B's scale to one
  int by_column;
  const float* master_in;
  float* master_out;            // NULL: not kept
  int64_t ld_master, batch_master;
  const uint8_t* g;             // the caller's G
  int64_t ld_g, batch_g;
  int g_dtype;
  uint8_t* y;                   // the caller's result in the last step, else NULL
  int64_t ld_y, batch_y;
  int y_dtype, y_wide, y_lines; // rows start on 16 bytes, on 32
  unsigned int* status;
  uint64_t timeout_ns;
  uint32_t debug_flags;
};

__device__ __forceinline__ uint32_t bf2_bits(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// tile t of the upper triangle of a grid with T columns, rows first; a row of
// tiles is as tall as R columns of them
__device__ __forceinline__ TileCoord upper_tile(uint32_t t, uint32_t T, uint32_t R) {
  uint32_t i = 0, left = t;
  while (left >= T - R * i) {
    left -= T - R * i;
    ++i;
  }
  TileCoord c;
  c.m = i;
  c.n = R * i + left;
  return c;
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                   const __grid_constant__ CUtensorMap tmB, const Params p) {
  using K_ = Cfg<BN, PAIR>;
  constexpr int CG = K_::CG, STAGES = K_::STAGES, KA = K_::KA, COLS = BN / K_::HALVES;
  constexpr uint32_t kTall = BN == 64 ? 2 : 1;  // rows of a tile, in its columns
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sA = ptx::smem_u32(smem);
  const uint32_t sB = sA + STAGES * K_::A_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * K_::STAGE_BYTES);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + K_::BARS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0);  // known uniform
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    ptx::prefetch_tensormap(&tmA);
    ptx::prefetch_tensormap(&tmB);
    for (uint32_t s = 0; s < uint32_t(STAGES); ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (uint32_t a = 0; a < 2; ++a) {
      ptx::mbar_init(tfull_bar(a), 1);
      ptx::mbar_init(tempty_bar(a), kEpiWarps / 2 * K_::HALVES * CG);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kEpiWarps + 1) {
    ptx::tmem_alloc<CG>(ptx::smem_u32(tmem_slot), 2 * BN);
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
  const uint32_t w0 = blockIdx.x / CG, P = gridDim.x / CG;
  const bool sym = p.mode != kUpdate;
  auto tile_at = [&](uint32_t w, uint32_t& b) -> TileCoord {
    b = w / p.per_matrix;
    const uint32_t t = w - b * p.per_matrix;
    return sym ? upper_tile(t, p.tiles_n, kTall) : tile_of(kSerpentine, t, p.tiles_m, p.tiles_n, 8u);
  };
  // nothing above touches global memory
  if (PAIR || warp >= kEpiWarps) ptx::grid_dep_wait();
  if (threadIdx.x == kEpiWarps * 32) ptx::grid_dep_launch_dependents();
  bool aborted = false;

  if (warp == kEpiWarps) {
    // ---------------- TMA producer ----------------
    // The whole warp runs the loop and one elected lane issues (also below):
    // descriptors and addresses then live in uniform registers.
    uint32_t stage = 0, phase = 0;
    bool skip = (p.debug_flags & SWZ_DEBUG_SKIP_FIRST_LOAD) != 0;
    const uint64_t pol = ptx::l2_policy_evict_last();
    const uint32_t full0 = PAIR ? ptx::map_to_rank(full_bar(0), 0) : full_bar(0);
    // R rows (or columns, MN-major) of an operand from r0, K elements k0 ..
    auto load = [&](auto rows, uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t r0,
                    int32_t k0, int32_t b, bool mn) {
      constexpr int R = decltype(rows)::value;
      if (mn) {
#pragma unroll
        for (int j = 0; j < R / 64; ++j) {
          if constexpr (PAIR)
            ptx::tma_load_3d_pair(dst + j * (64 * KA * 128), map, bar, r0 + 64 * j, k0, b, pol);
          else
            ptx::tma_load_3d(dst + j * (64 * KA * 128), map, bar, r0 + 64 * j, k0, b, pol);
        }
      } else {
#pragma unroll
        for (int j = 0; j < KA; ++j) {
          if constexpr (PAIR)
            ptx::tma_load_3d_pair(dst + j * (R * 128), map, bar, k0 + 64 * j, r0, b, pol);
          else
            ptx::tma_load_3d(dst + j * (R * 128), map, bar, k0 + 64 * j, r0, b, pol);
        }
      }
    };
    const std::integral_constant<int, BM> a_rows;
    const std::integral_constant<int, K_::BN_LOCAL> b_rows;
    for (uint32_t w = w0; w < p.units && !aborted; w += P) {
      uint32_t b;
      const TileCoord t = tile_at(w, b);
      const int32_t m0 = int32_t((t.m * CG + rank) * BM);
      const int32_t n0 = int32_t(t.n * BN + rank * K_::BN_LOCAL);
      for (uint32_t kb = 0; kb < p.num_kb; ++kb) {
        const bool ok = pipe::wait(empty_bar(stage), phase ^ 1u, ctl);
        if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
        if (pipe::elect_one()) {
          if (leader) ptx::mbar_arrive_expect_tx(full_bar(stage), CG * K_::STAGE_BYTES);
          if (!skip) {
            const int32_t k0 = int32_t(kb * (64 * KA));
            load(a_rows, sA + stage * K_::A_BYTES, &tmA, full0 + 8u * stage, m0, k0, int32_t(b),
                 p.a_mn != 0);
            load(b_rows, sB + stage * K_::B_BYTES, &tmB, full0 + 8u * stage, n0, k0, int32_t(b),
                 p.b_mn != 0);
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
  } else if (warp == kEpiWarps + 1) {
    // ---------------- MMA issuer (leader CTA) ----------------
    if (leader) {
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool issued = false;
      const uint64_t adesc0 = p.a_mn ? pipe::sdesc128(sA, 64 * KA * 128, 1024)
                                     : pipe::sdesc128(sA, 16, 1024);
      const uint64_t bdesc0 = p.b_mn ? pipe::sdesc128(sB, 64 * KA * 128, 1024)
                                     : pipe::sdesc128(sB, 16, 1024);
      const bool amn = p.a_mn != 0, bmn = p.b_mn != 0;
      for (uint32_t w = w0; w < p.units && !aborted; w += P) {
        bool ok = pipe::wait(tempty_bar(acc), acc_phase ^ 1u, ctl);
        if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + acc * BN;
        for (uint32_t kb = 0; kb < p.num_kb; ++kb) {
          ok = pipe::wait(full_bar(stage), phase, ctl);
          if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
          ptx::tc_fence_after();
          const uint64_t a = adesc0 + uint64_t(stage * uint32_t(K_::A_BYTES >> 4));
          const uint64_t b = bdesc0 + uint64_t(stage * uint32_t(K_::B_BYTES >> 4));
          if (pipe::elect_one()) {
            // slice kk: 16 elements of K; K-major 32 bytes into atom kk / 4,
            // MN-major 16 rows of 128 bytes down
#pragma unroll
            for (uint32_t kk = 0; kk < uint32_t(4 * KA); ++kk) {
              const uint32_t ka_at = ((kk / 4) * (BM * 128) + (kk % 4) * 32) >> 4;
              const uint32_t kb_at = ((kk / 4) * (K_::BN_LOCAL * 128) + (kk % 4) * 32) >> 4;
              const uint32_t mn = 128u * kk;
              ptx::mma<CG, 0>(d, a + (amn ? mn : ka_at), b + (bmn ? mn : kb_at), p.idesc,
                              kb != 0 || kk != 0);
            }
            if constexpr (PAIR) ptx::mma_commit_pair(empty_bar(stage), 0x3);
            else ptx::mma_commit(empty_bar(stage));
            if (kb + 1 == p.num_kb) {
              if constexpr (PAIR) ptx::mma_commit_pair(tfull_bar(acc), 0x3);
              else ptx::mma_commit(tfull_bar(acc));
            }
          }
          __syncwarp();
          issued = true;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (aborted && issued) {
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
    // ---------------- epilogue ----------------
    // A warp takes 32 rows and 64 columns at a time.  What the sums are added
    // to is loaded before the tile's products are waited for: a chunk's loads
    // after the wait cost an L2 round trip each, most of a small product's time.
    // Of 64-wide tiles warps 0-3 take every other one, 4-7 the rest.
    const uint32_t q = warp & 3u, half = warp >> 2;
    const uint32_t half_col = K_::HALVES == 2 ? half * COLS : 0u;
    uint32_t acc = 0, acc_phase = 0;
    // A single CTA's warps run their code once before they wait for the kernel
    // before, with rows past the end, so that nothing is loaded or stored: its
    // instructions then need not be fetched at the first tile's end (512 x 512
    // 83 us, 91 without; 1024 x 1024 112 and 119; pairs are 1 % slower with it).
    bool warm = !PAIR;
    for (uint32_t w = w0; warm || (w < p.units && !aborted);) {
      if (K_::HALVES == 1 && !warm && acc != half) {
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
        w += P;
        continue;
      }
      uint32_t b;
      const TileCoord t = tile_at(w, b);
      const int64_t row = (warm ? int64_t(p.tiles_m) : int64_t(t.m)) * (CG * BM) + rank * BM +
                          q * 32 + lane;
      const bool row_in = row < p.M;
      // rows of 128 bytes as a warp loads and stores them (quad_transpose)
      const int64_t line0 = row - lane + (lane / 4) * 4;
      const uint32_t piece = lane % 4;
      Scale sc = {};
      if (!warm) sc = p.scale[b];
      const float fx = p.first ? sc.f : sc.down;  // X over the fp16 X's power of two
      const float f = p.mode == kPoly ? p.f : p.mode == kGram ? p.f * fx * fx : p.f * fx;
      const float out_scale = p.mode == kUpdate ? p.out_scale * sc.up : 1.f;
      // of a X: by row, or (1 here) below by column
      const float* const factor = p.factor + b * p.batch_factor;
      float a = 1.f;
      if (p.mode == kUpdate && !p.by_column && row_in) a = factor[row];
      const float u16 = p.mode == kPoly ? p.u : a * p.u * fx;
#pragma unroll 1
      for (int h = 0; h < COLS / 64; ++h) {
        const int64_t col0 = int64_t(t.n) * BN + half_col + h * 64;
        float v[64];
        const bool by_column = p.mode == kUpdate && p.by_column && !warm;
        float f0 = 0.f, f1 = 0.f;
        if (by_column) {
          if (col0 + lane < p.N) f0 = factor[col0 + lane];
          if (col0 + 32 + lane < p.N) f1 = factor[col0 + 32 + lane];
        }
        if (p.mode == kGram) {
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] = 0.f;
        } else if (p.mode == kPoly || p.source == kFromF16) {
          uint32_t x[32];
          const __half* src = p.in + b * p.batch_in + line0 * p.ld_in + col0 + piece * 16;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[8 * j + k] = 0u;
            if (line0 + j < p.M && col0 + piece * 16 < p.N)
              pipe::ld_global_8(src + j * p.ld_in, x + 8 * j);
          }
          pipe::quad_transpose(x, lane);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
            v[2 * j] = u16 * z.x;
            v[2 * j + 1] = u16 * z.y;
          }
        } else if (p.source == kFromF32) {
          const float* src = p.master_in + b * p.batch_master + line0 * p.ld_master + col0 + piece * 8;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int k = 0; k < 8; ++k) x[8 * j + k] = 0u;
              if (line0 + j < p.M && col0 + c * 32 + piece * 8 < p.N)
                pipe::ld_global_8(src + j * p.ld_master + c * 32, x + 8 * j);
            }
            pipe::quad_transpose(x, lane);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[c * 32 + j] = a * __uint_as_float(x[j]);
          }
        } else {
          // G, or its fp32 copy: whole lines, one of 16-bit values, two of fp32
          const float g1 = a * sc.p1, g2 = sc.p2 * sc.f;
          const int es = p.g_dtype == SWZ_F32 ? 4 : 2;
          const uint8_t* src =
              p.g + (b * p.batch_g + line0 * p.ld_g + col0) * es + piece * 32;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c == 1 && es == 2) break;
            const int64_t col = col0 + (es == 4 ? c * 32 + piece * 8 : piece * 16);
            uint32_t x[32];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int k = 0; k < 8; ++k) x[8 * j + k] = 0u;
              if (line0 + j < p.M && col < p.N)
                pipe::ld_global_8(src + j * p.ld_g * es + c * 128, x + 8 * j);
            }
            pipe::quad_transpose(x, lane);
            if (es == 4) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[c * 32 + j] = __uint_as_float(x[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                v[j] = p.g_dtype == SWZ_BF16 ? f8::Bf16::value(x, j) : f8::F16::value(x, j);
            }
          }
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] = v[j] * g1 * g2;
        }
        if (by_column) {
          // a lane holds the factors of two columns
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            v[j] *= __shfl_sync(0xFFFFFFFFu, f0, j);
            v[32 + j] *= __shfl_sync(0xFFFFFFFFu, f1, j);
          }
        }
        if (h == 0 && !warm) {
          const bool ok = pipe::wait(tfull_bar(acc), acc_phase, ctl);
          if (!__all_sync(0xFFFFFFFFu, ok)) { aborted = true; break; }
          ptx::tc_fence_after();
        }
        __syncwarp();
        const uint32_t taddr = tmem_base + ((q * 32u) << 16) + acc * BN + half_col + h * 64;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[32];
          ptx::tmem_ld_32x32b_x32(taddr + c * 32, r);
          pipe::tmem_ld_wait32(r);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[c * 32 + j] = fmaf(f, __uint_as_float(r[j]), v[c * 32 + j]);
        }
        if (h + 1 == COLS / 64) {  // the tile is in registers
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0 && !warm) {
            if constexpr (PAIR) pipe::arrive_at(ptx::map_to_rank(tempty_bar(acc), 0));
            else ptx::mbar_arrive(tempty_bar(acc));
          }
        }
        if (p.y) {
          // the result: rows that start on 16 bytes by the row, others with a
          // lane a column
          const int es = p.y_dtype == SWZ_F32 ? 4 : 2;
          uint8_t* y = p.y + (b * p.batch_y) * es;
          if (p.y_lines && col0 + 64 <= p.N) {
            uint8_t* to = y + (line0 * p.ld_y + col0) * es + piece * 32;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (c == 1 && es == 2) break;
              uint32_t x[32];
              if (es == 4) {
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(v[c * 32 + j]);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  x[j] = p.y_dtype == SWZ_BF16 ? bf2_bits(v[2 * j], v[2 * j + 1])
                                               : half2_bits(v[2 * j], v[2 * j + 1]);
              }
              pipe::quad_transpose(x, lane);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (line0 + j < p.M) pipe::st_global_32b(to + j * p.ld_y * es + c * 128, x + 8 * j);
            }
          } else if (p.y_wide) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int64_t col = col0 + c * 8;
              if (!row_in || col >= p.N) continue;
              uint8_t* to = y + (row * p.ld_y + col) * es;
              const float* x = v + c * 8;
              if (col + 8 > p.N) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (col + j < p.N) store_any(to, j, x[j], p.y_dtype);
              } else if (p.y_dtype == SWZ_F32) {
                reinterpret_cast<float4*>(to)[0] = make_float4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<float4*>(to)[1] = make_float4(x[4], x[5], x[6], x[7]);
              } else {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  o[j] = p.y_dtype == SWZ_BF16 ? bf2_bits(x[2 * j], x[2 * j + 1])
                                               : half2_bits(x[2 * j], x[2 * j + 1]);
                *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float x[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = v[c * 32 + i];
              pipe::transpose32(x, lane);
              const int64_t col = col0 + c * 32 + lane, r0 = row - lane;
              if (col < p.N)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (r0 + i < p.M) store_any(y, (r0 + i) * p.ld_y + col, x[i], p.y_dtype);
              __syncwarp();
            }
          }
          continue;
        }
        if (p.master_out) {
          float* dst = p.master_out + b * p.batch_master + line0 * p.ld_master + col0 + piece * 8;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(v[c * 32 + j]);
            pipe::quad_transpose(x, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (line0 + j < p.M && col0 + c * 32 + piece * 8 < p.N)
                pipe::st_global_32b(dst + j * p.ld_master + c * 32, x + 8 * j);
          }
        }
        uint32_t o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
          o[j] = half2_bits(v[2 * j] * out_scale, v[2 * j + 1] * out_scale);
        __half* out = p.out + b * p.batch_out;
        if (p.mode == kPoly && row - lane >= col0 && row - lane < col0 + 64) {
          // this warp's piece of the diagonal: column `lane` of one half
          const bool second = row - lane != col0;
          float z = 0.f;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float e = second ? v[32 + j] : v[j];
            const uint32_t two = second ? o[16 + j / 2] : o[j / 2];
            const float rounded =
                __half2float(__ushort_as_half(uint16_t((j & 1) ? two >> 16 : two)));
            z = int(lane) == j ? e - rounded : z;
          }
          if (row_in) p.factor[b * p.batch_factor + row] = fmaf(p.lost_scale, z, p.a);
        }
        if (sym && t.m != t.n / kTall) {
          // The other half: lanes are neighbours along its rows.  Two lanes
          // swap a value of each column pair, so that each stores two rows'
          // values of one of the columns (one value a store took twice as long)
          __half* const to = out + (col0 + (lane & 1u)) * p.ld_out + (row & ~int64_t(1));
          const bool in = (row & ~int64_t(1)) < p.M;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint32_t got =
                __shfl_xor_sync(0xFFFFFFFFu, (lane & 1u) ? o[k] & 0xFFFFu : o[k] >> 16, 1);
            const uint32_t two = (lane & 1u) ? got | (o[k] & 0xFFFF0000u)
                                             : (o[k] & 0xFFFFu) | (got << 16);
            if (in && col0 + 2 * k + (lane & 1u) < p.N)
              *reinterpret_cast<uint32_t*>(to + 2 * k * p.ld_out) = two;
          }
        }
        __syncwarp();
        pipe::quad_transpose(o, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (line0 + j < p.M && col0 + piece * 16 < p.N)
            pipe::st_global_32b(out + (line0 + j) * p.ld_out + col0 + piece * 16, o + 8 * j);
      }
      if (warm) {
        warm = false;
        ptx::grid_dep_wait();
        continue;
      }
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
      w += P;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp == kEpiWarps + 1) ptx::tmem_dealloc<CG>(tmem_base, 2 * BN);
}

// ---- the norm and the first X ---------------------------------------------------
// Sum of squares of each matrix in three scales -- as they are, and of the
// values times 2^-80 and 2^80 -- so that no finite G overflows and none that
// matters underflows; per CTA in fp32 by thread, then in double, in a fixed
// order.
constexpr int kNormThreads = 256, kNormUnroll = 4;

struct NormArgs {
  const uint8_t* g;
  int64_t ld_g, batch_g;
  int g_dtype, m, n;
  int wide;              // rows of G start on 16 bytes
  uint32_t parts;        // CTAs of a matrix
  double* partial;       // [batch][parts][3]
  double eps;
  double headroom;       // see make_scale
  Scale* scale;
  __half* x;             // first fp16 X
  float* g32;            // a copy of G, or NULL; both rows as X's
  int64_t ld_x, batch_x;
};

template <typename T>
__global__ void __launch_bounds__(kNormThreads) ns_norm_kernel(const NormArgs p) {
  __shared__ double red[3][kNormThreads / 32];
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t b = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const uint32_t chunks = (uint32_t(p.n) + 7u) / 8u;  // of 8 values of a row
  const uint32_t total = chunks * uint32_t(p.m);      // at most 2^28 + m
  const uint32_t beg = uint32_t(uint64_t(total) * part / p.parts);
  const uint32_t end = uint32_t(uint64_t(total) * (part + 1) / p.parts);
  const uint8_t* g = p.g + b * p.batch_g * T::kBytes;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f;
#pragma unroll 1
  for (uint32_t i0 = beg + threadIdx.x; i0 < end; i0 += kNormThreads * kNormUnroll) {
    uint32_t w[kNormUnroll][T::kWords];
#pragma unroll
    for (int k = 0; k < kNormUnroll; ++k) {
      const uint32_t i = i0 + k * kNormThreads, r = i / chunks, c = i - r * chunks;
      f8::load8<T>(g + (int64_t(r) * p.ld_g + c * 8) * T::kBytes,
                   i < end ? p.n - int(c * 8) : 0, p.wide != 0, w[k]);
    }
#pragma unroll
    for (int k = 0; k < kNormUnroll; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = T::value(w[k], j), lo = v * 0x1p-80f, hi = v * 0x1p80f;
        s0 = fmaf(v, v, s0);
        s1 = fmaf(lo, lo, s1);
        s2 = fmaf(hi, hi, s2);
      }
  }
  double d[3] = {s0, s1, s2};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) d[k] += __shfl_xor_sync(0xFFFFFFFFu, d[k], o);
    if (threadIdx.x % 32 == 0) red[k][threadIdx.x / 32] = d[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    double v = 0.0;
    for (int j = 0; j < kNormThreads / 32; ++j) v += red[threadIdx.x][j];
    p.partial[(uint64_t(b) * p.parts + part) * 3 + threadIdx.x] = v;
  }
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) ns_start_kernel(const NormArgs p) {
  __shared__ Scale sc;
  ptx::grid_dep_wait();
  if (threadIdx.x == 0) ptx::grid_dep_launch_dependents();
  const uint32_t b = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  if (threadIdx.x < 32) {
    double d[3] = {0.0, 0.0, 0.0};
    for (uint32_t j = threadIdx.x; j < p.parts; j += 32)
#pragma unroll
      for (int k = 0; k < 3; ++k) d[k] += p.partial[(uint64_t(b) * p.parts + j) * 3 + k];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int o = 16; o > 0; o /= 2) d[k] += __shfl_xor_sync(0xFFFFFFFFu, d[k], o);
    if (threadIdx.x == 0) {
      sc = make_scale(d, double(p.m) * double(p.n), p.eps, p.headroom);
      if (part == 0) p.scale[b] = sc;
    }
  }
  __syncthreads();
  const float p1 = sc.p1, p2 = sc.p2;
  const uint32_t chunks = (uint32_t(p.n) + 7u) / 8u;
  const uint32_t total = chunks * uint32_t(p.m);
  const uint32_t beg = uint32_t(uint64_t(total) * part / p.parts);
  const uint32_t end = uint32_t(uint64_t(total) * (part + 1) / p.parts);
  const uint8_t* g = p.g + b * p.batch_g * T::kBytes;
  __half* x = p.x + b * p.batch_x;
#pragma unroll 1
  for (uint32_t i0 = beg + threadIdx.x; i0 < end; i0 += kNormThreads * kNormUnroll) {
    uint32_t w[kNormUnroll][T::kWords];
#pragma unroll
    for (int k = 0; k < kNormUnroll; ++k) {
      const uint32_t i = i0 + k * kNormThreads, r = i / chunks, c = i - r * chunks;
      f8::load8<T>(g + (int64_t(r) * p.ld_g + c * 8) * T::kBytes,
                   i < end ? p.n - int(c * 8) : 0, p.wide != 0, w[k]);
    }
#pragma unroll
    for (int k = 0; k < kNormUnroll; ++k) {
      const uint32_t i = i0 + k * kNormThreads, r = i / chunks, c = i - r * chunks;
      if (i >= end) continue;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = half2_bits(T::value(w[k], 2 * j) * p1 * p2, T::value(w[k], 2 * j + 1) * p1 * p2);
      *reinterpret_cast<uint4*>(x + int64_t(r) * p.ld_x + c * 8) =
          make_uint4(o[0], o[1], o[2], o[3]);
      if (p.g32) {
        float4* to = reinterpret_cast<float4*>(p.g32 + b * p.batch_x + int64_t(r) * p.ld_x + c * 8);
        to[0] = make_float4(T::value(w[k], 0), T::value(w[k], 1), T::value(w[k], 2),
                            T::value(w[k], 3));
        to[1] = make_float4(T::value(w[k], 4), T::value(w[k], 5), T::value(w[k], 6),
                            T::value(w[k], 7));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static uint64_t round_up(uint64_t a, uint64_t b) { return (a + b - 1) / b * b; }

constexpr uint32_t kMaxParts = 1024;  // CTAs that share a matrix's norm

struct Layout {
  int64_t ldx, ldd;                        // elements
  uint64_t x0, x1, master, a, b, factor, partial, scale, total;  // byte offsets
};

static Layout layout(uint64_t batch, uint64_t m, uint64_t n) {
  const uint64_t d = m < n ? m : n;
  Layout L;
  L.ldx = int64_t(round_up(n, 16));
  L.ldd = int64_t(round_up(d, 16));
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  L.x0 = take(batch * m * L.ldx * 2);
  L.x1 = take(batch * m * L.ldx * 2);
  L.master = take(batch * m * L.ldx * 4);
  L.a = take(batch * d * L.ldd * 2);
  L.b = take(batch * d * L.ldd * 2);
  L.factor = take(batch * L.ldd * 4);
  L.partial = take(batch * kMaxParts * 3 * 8);
  L.scale = take(batch * sizeof(Scale));
  L.total = at;
  return L;
}

// largest |a s + b s^3 + c s^5| on [0, hi]
static double poly_max(double a, double b, double c, double hi) {
  auto at = [&](double s) { return fabs(s * (a + s * s * (b + c * s * s))); };
  double best = at(hi);
  // where the derivative a + 3 b t + 5 c t^2 vanishes, t = s^2
  const double disc = 9 * b * b - 20 * a * c;
  double t[3] = {-1, -1, -1};
  if (c != 0 && disc >= 0) {
    t[0] = (-3 * b + sqrt(disc)) / (10 * c);
    t[1] = (-3 * b - sqrt(disc)) / (10 * c);
  } else if (c == 0 && b != 0) {
    t[2] = -a / (3 * b);
  }
  for (double x : t)
    if (x > 0 && x < hi * hi) best = fmax(best, at(sqrt(x)));
  return best;
}

// exponent of the largest power of two that keeps values up to `bound` below
// 2^15 in fp16, between -100 and `most`
static int room(double bound, int most) {
  if (!(bound > 0)) return most;
  const int e = 14 - int(ceil(log2(bound)));
  return e < -100 ? -100 : e > most ? most : e;
}

template <int BN, bool PAIR>
static int launch(const CUtensorMap& ta, const CUtensorMap& tb, const Params& prm, int num_sms,
                  cudaStream_t stream) {
  using K_ = Cfg<BN, PAIR>;
  auto kern = ns_gemm_kernel<BN, PAIR>;
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
  const uint32_t cap = uint32_t(num_sms) / K_::CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((prm.units < cap ? prm.units : cap) * K_::CG);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = K_::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = K_::CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, ta, tb, prm));
  return SWZ_OK;
}

template <typename T>
static int launch_norm(const NormArgs& a, uint32_t grid, bool start, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kNormThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (start) SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, ns_start_kernel<T>, a));
  else SWZ_CUDA_TRY(cudaLaunchKernelEx(&cfg, ns_norm_kernel<T>, a));
  return SWZ_OK;
}

struct Operand {
  const __half* p;
  uint64_t rows, cols;
  int64_t ld;
  bool mn;  // given K x rows
};

// tiles of an M x N product in tiles of a rows and b columns (a a multiple of b)
static uint64_t tiles_of(uint64_t M, uint64_t N, bool sym, uint64_t a, uint64_t b) {
  const uint64_t tm = (M + a - 1) / a, tn = (N + b - 1) / b;
  return sym ? tm * tn - a / b * (tm * (tm - 1) / 2) : tm * tn;
}

// The width of the tiles that all products of a call take: 256 (CTA pairs), 128
// or 64, by the estimated time of a step in us -- for each product a fixed part,
// then for each wave of tiles its stages of K, or its epilogue where that is
// longer.  128-wide tiles read 64 KB for 128 of K, 64-wide ones 48 KB, which is
// what bounds them.  Whole calls, fp32, five steps, us with 64 / 128 / 256: 512 x
// 512 90 / 104 / 168, 1024 x 1024 118 / 131 / 202, 600 x 4000 174 / 195 / 255, 2048 x
// 2048 312 / 238 / 288, 2500 x 2500 559 / 474 / 411, 4096 x 4096 1694 / 1243 / 952.
// One shape for all three products: a kernel that follows another one in
// the stream starts about 2.5 us later than one that follows itself, and every
// mixture measured was slower.
static int width_for(uint64_t batch, uint64_t d, uint64_t len, bool wide, uint64_t sms) {
  struct Shape {
    int width;
    uint64_t rows, ctas;
    double fixed, stage, epilogue;
  };
  const Shape shapes[3] = {
      {64, 128, 1, 4.0, 0.39, 1.1}, {128, 128, 1, 4.0, 0.53, 2.2}, {256, 256, 2, 8.7, 0.64, 4.4}};
  int best = 0;
  double least = 0;
  for (const Shape& s : shapes) {
    double t = 0;
    for (int product = 0; product < 3; ++product) {  // A, B, the new X
      const bool sym = product < 2;
      const uint64_t K = product == 0 ? len : d;
      const uint64_t M = sym || wide ? d : len, N = sym || !wide ? d : len;
      const uint64_t tiles = batch * tiles_of(M, N, sym, s.rows, uint64_t(s.width));
      const uint64_t at_once = sms / s.ctas;
      t += s.fixed + double((tiles + at_once - 1) / at_once) *
                         fmax(s.stage * double((K + 127) / 128), s.epilogue);
    }
    if (best == 0 || t < least) {
      best = s.width;
      least = t;
    }
  }
  return best;
}

// One product: the maps and the launch.
static int product(const Operand& A, const Operand& B, uint64_t batch, uint64_t K, Params prm,
                   const DeviceInfo& dev, int width, cudaStream_t s) {
  const uint64_t M = uint64_t(prm.M), N = uint64_t(prm.N);
  const bool sym = prm.mode != kUpdate;
  const bool pair = width == 256;
  const uint64_t bm = pair ? 256 : 128, bn = uint64_t(width);
  const int ka = pair ? 1 : 2;
  CUtensorMap map[2];
  const Operand* ops[2] = {&A, &B};
  for (int i = 0; i < 2; ++i) {
    const Operand& o = *ops[i];
    const int rc = encode_half(&map[i], o.p, batch, o.rows, o.cols, uint64_t(o.ld),
                               o.rows * uint64_t(o.ld), 64,
                               o.mn ? 64u * ka : i == 1 && width == 64 ? 64u : 128u);
    if (rc != SWZ_OK) return rc;
  }
  const uint64_t units = batch * tiles_of(M, N, sym, bm, bn);
  if (units > uint64_t(INT32_MAX)) return SWZ_EINVAL;
  prm.tiles_m = uint32_t((M + bm - 1) / bm);
  prm.tiles_n = uint32_t((N + bn - 1) / bn);
  prm.units = uint32_t(units);
  prm.per_matrix = uint32_t(units / batch);
  prm.num_kb = uint32_t((K + 64 * ka - 1) / (64 * ka));
  prm.a_mn = A.mn;
  prm.b_mn = B.mn;
  prm.idesc = pipe::idesc(0, 0, A.mn, B.mn, int(bm), int(bn));
  if (width == 64) return launch<64, false>(map[0], map[1], prm, dev.num_sms, s);
  return pair ? launch<256, true>(map[0], map[1], prm, dev.num_sms, s)
              : launch<128, false>(map[0], map[1], prm, dev.num_sms, s);
}

}  // namespace ns
}  // namespace swz

using namespace swz;
using namespace swz::ns;

static bool sizes_ok(int batch, int m, int n) {
  return batch >= 0 && m >= 0 && n >= 0 && int64_t(m) * n <= (int64_t(1) << 31) && batch <= 65535;
}

// True when a value of Y may lie where another one of G is: each matrix and each
// tile reads its own values of G before it writes them, but not another's.  The
// ranges of views that share rows without sharing columns meet, their values do
// not.
static bool lies_across(uintptr_t ga, int64_t gs, int64_t ldg, int64_t bsg, uintptr_t ya,
                        int64_t ys, int64_t ldy, int64_t bsy, int batch, int m, int n) {
  auto bytes = [&](int64_t es, int64_t ld, int64_t bs) {
    return uintptr_t(((batch - 1) * bs + (m - 1) * ld + n) * es);
  };
  if (ga >= ya + bytes(ys, ldy, bsy) || ya >= ga + bytes(gs, ldg, bsg)) return false;
  if (gs != ys || (m > 1 && ldg != ldy) || (batch > 1 && bsg != bsy)) return true;
  if (ga == ya) return false;
  const int64_t d = ya > ga ? int64_t(ya - ga) : int64_t(ga - ya);
  if (m == 1 || d % gs != 0 || (batch > 1 && bsg % ldg != 0)) return true;
  const int64_t column = d / gs % ldg;
  return column < n || column + n > ldg;
}

extern "C" int swz_newton_schulz_workspace_size(int batch, int m, int n, uint64_t* h_bytes) {
  if (!h_bytes || !sizes_ok(batch, m, n)) return SWZ_EINVAL;
  *h_bytes = batch && m && n ? layout(uint64_t(batch), uint64_t(m), uint64_t(n)).total : 0;
  return SWZ_OK;
}

extern "C" int swz_newton_schulz(const void* G, int dtype, int64_t ldg, int64_t batch_stride_g,
                                 void* Y, int y_dtype, int64_t ldy, int64_t batch_stride_y,
                                 int batch, int m, int n, int steps, double a, double b, double c,
                                 double eps, const swz_newton_schulz_opts* opts, void* d_workspace,
                                 uint64_t workspace_bytes, void* stream) {
  swz_newton_schulz_opts o = {};
  if (opts) o = *opts;
  if (!sizes_ok(batch, m, n) || steps < 1 || steps > kMaxSteps) return SWZ_EINVAL;
  for (int d : {dtype, y_dtype})
    if (d != SWZ_F16 && d != SWZ_BF16 && d != SWZ_F32) return SWZ_EINVAL;
  if (!(eps >= 0.0) || !isfinite(eps) || !isfinite(a) || !isfinite(b) || !isfinite(c))
    return SWZ_EINVAL;
  if (o.tile != 0 && o.tile != 128 && o.tile != 256) return SWZ_EUNSUPPORTED;
  if (batch == 0 || m == 0 || n == 0) return SWZ_OK;
  const int64_t gs = dtype == SWZ_F32 ? 4 : 2, ys = y_dtype == SWZ_F32 ? 4 : 2;
  const uintptr_t ga = reinterpret_cast<uintptr_t>(G);
  if (!G || ga % uintptr_t(gs) != 0 || (m > 1 && ldg < n) ||
      (batch > 1 && batch_stride_g < (m - 1) * ldg + n))
    return SWZ_EINVAL;
  const uintptr_t ya = reinterpret_cast<uintptr_t>(Y);
  if (!Y || ya % uintptr_t(ys) != 0 || (m > 1 && ldy < n) ||
      (batch > 1 && batch_stride_y < (m - 1) * ldy + n))
    return SWZ_EINVAL;
  // the range of singular values, step by step, gives the powers of two
  // and how far below them X can stay: hi over the largest growth, in all steps
  double hi[kMaxSteps + 1], grown = 1.0, headroom = 1.0;
  hi[0] = 1.0;
  for (int i = 0; i < steps; ++i) {
    hi[i + 1] = 1.01 * poly_max(a, b, c, hi[i]);
    if (!(hi[i + 1] < 1e15)) return SWZ_EUNSUPPORTED;
    const double h2 = hi[i] * hi[i], mid = c != 0 ? -b / (2 * c) : -1.0;
    double g = fmax(fabs(a), fabs(a + h2 * (b + c * h2)));
    if (mid > 0 && mid < h2) g = fmax(g, fabs(a + mid * (b + c * mid)));
    grown *= 1.01 * g;
    if (grown > 0) headroom = fmin(headroom, hi[i + 1] / grown);
  }
  // powers of two that keep X, A and B in the range of fp16, by step
  int ex[kMaxSteps], ea[kMaxSteps], eb[kMaxSteps];
  for (int i = 0; i < steps; ++i) {
    const double h2 = hi[i] * hi[i] * 1.01;
    ex[i] = i == 0 ? 0 : room(hi[i] * 1.01, 12);  // the first X goes by its Scale
    ea[i] = room(h2, 14);
    // largest |b t + c t^2| on [0, h2]
    double bmax = fabs(h2 * (b + c * h2));
    if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < h2) bmax = fmax(bmax, b * b / (4 * fabs(c)));
    eb[i] = room(1.01 * bmax, 14);
  }
  const Layout L = layout(uint64_t(batch), uint64_t(m), uint64_t(n));
  const uintptr_t wsa = reinterpret_cast<uintptr_t>(d_workspace);
  if (!wsa || (wsa & 255u) || workspace_bytes < L.total) return SWZ_EINVAL;
  DeviceInfo dev{};
  int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  const uint64_t timeout_ns = uint64_t(o.timeout_ms ? o.timeout_ms : 2000u) * 1000000ull;
  const bool wide = m <= n;
  const uint64_t d = uint64_t(wide ? m : n);

  // Where Y lies across G, G has to be read before any of Y is written.  The
  // kernels of their own do so but when their only update reads G itself, the one
  // kernel when there is no other matrix.
  const bool across = lies_across(ga, gs, ldg, batch_stride_g, ya, ys, ldy, batch_stride_y, batch,
                                  m, n);
  bool small = o.tile == 0 && d <= kSmallSide && (wide ? n : m) <= kSmallLong &&
               !(across && batch > 1);
  if (small) {
    rc = small_pays(batch, wide ? n : m, &small);
    if (rc != SWZ_OK) return rc;
  }
  if (small) {
    SmallParams p{};
    p.g = static_cast<const uint8_t*>(G);
    p.ld_g = m > 1 ? ldg : n;
    p.batch_g = batch > 1 ? batch_stride_g : 0;
    p.g_dtype = dtype;
    p.y = static_cast<uint8_t*>(Y);
    p.ld_y = m > 1 ? ldy : n;
    p.batch_y = batch > 1 ? batch_stride_y : 0;
    p.y_dtype = y_dtype;
    p.wide = wide;
    p.d = int(d);
    p.len = wide ? n : m;
    p.steps = steps;
    p.eps = eps;
    p.headroom = headroom;
    p.debug_flags = o.debug_flags;
    p.timeout_ns = timeout_ns;
    rc = op_status_word(&p.status);
    if (rc != SWZ_OK) return rc;
    for (int i = 0; i < steps; ++i) {
      p.fa[i] = float(exp2(double(ea[i] - 2 * ex[i])));
      p.ub[i] = float(b * exp2(double(eb[i] - ea[i])));
      p.fb[i] = float(c * exp2(double(eb[i] - 2 * ea[i])));
      p.k1[i] = float(exp2(double(-eb[i] - ex[i])));
      p.sx[i] = float(exp2(double(ex[i])));
      p.ad[i] = float(a * exp2(double(eb[i])));
    }
    return launch_small(p, batch, s);
  }

  NormArgs na{};
  na.g = static_cast<const uint8_t*>(G);
  na.ld_g = m > 1 ? ldg : n;
  na.batch_g = batch > 1 ? batch_stride_g : 0;
  na.g_dtype = dtype;
  na.m = m;
  na.n = n;
  na.wide = ga % 16 == 0 && (m == 1 || (na.ld_g * gs) % 16 == 0) &&
            (batch == 1 || (na.batch_g * gs) % 16 == 0);
  // no more CTAs than fill the GPU
  const uint64_t chunks = (uint64_t(n) + 7) / 8 * uint64_t(m);
  uint64_t parts = (chunks + 1023) / 1024;  // one round of kNormUnroll chunks a thread
  const uint64_t fill = (uint64_t(dev.num_sms) * 4 + batch - 1) / batch;
  if (parts > fill) parts = fill;
  if (parts > kMaxParts) parts = kMaxParts;
  na.parts = uint32_t(parts);
  na.partial = reinterpret_cast<double*>(ws + L.partial);
  na.eps = eps;
  na.headroom = headroom;
  na.scale = reinterpret_cast<Scale*>(ws + L.scale);
  na.x = reinterpret_cast<__half*>(ws + L.x0);
  // The first update reads G by whole lines of 64 values.  Rows that do not start
  // on 16 bytes or are no multiple of a line it reads from an fp32 copy, which is
  // left where the fp32 X will be.  Element by element in its epilogue it took 49
  // us instead of 15 at 1001 x 1001, 129 instead of 28 for 14 of 2533 x 199.
  const bool lines = na.wide && n % 64 == 0 && !(across && steps == 1);
  na.g32 = lines ? nullptr : reinterpret_cast<float*>(ws + L.master);
  na.ld_x = L.ldx;
  na.batch_x = int64_t(m) * L.ldx;
  const uint32_t grid = uint32_t(parts) * uint32_t(batch);
  for (int start = 0; start < 2; ++start) {
    if (dtype == SWZ_BF16) rc = launch_norm<f8::Bf16>(na, grid, start != 0, s);
    else if (dtype == SWZ_F16) rc = launch_norm<f8::F16>(na, grid, start != 0, s);
    else rc = launch_norm<f8::F32>(na, grid, start != 0, s);
    if (rc != SWZ_OK) return rc;
  }

  Params base{};
  base.g = lines ? na.g : reinterpret_cast<const uint8_t*>(na.g32);
  base.ld_g = lines ? na.ld_g : L.ldx;
  base.batch_g = lines ? na.batch_g : int64_t(m) * L.ldx;
  base.g_dtype = lines ? dtype : int(SWZ_F32);
  base.ld_master = L.ldx;
  base.batch_master = int64_t(m) * L.ldx;
  base.timeout_ns = timeout_ns;
  base.debug_flags = o.debug_flags;
  base.scale = na.scale;
  base.factor = reinterpret_cast<float*>(ws + L.factor);
  base.batch_factor = L.ldd;
  base.by_column = !wide;
  rc = op_status_word(&base.status);
  if (rc != SWZ_OK) return rc;
  __half* const xs[2] = {reinterpret_cast<__half*>(ws + L.x0),
                         reinterpret_cast<__half*>(ws + L.x1)};
  __half* const Am = reinterpret_cast<__half*>(ws + L.a);
  __half* const Bm = reinterpret_cast<__half*>(ws + L.b);
  float* const master = reinterpret_cast<float*>(ws + L.master);
  const int width = o.tile ? o.tile
                           : width_for(uint64_t(batch), d, uint64_t(wide ? n : m), wide,
                                       uint64_t(dev.num_sms));
  // steps that take the a X term in fp32 (the first takes G itself in any case)
  const int masters = steps - 2;
  for (int i = 0; i < steps; ++i) {
    __half* const x = xs[i & 1];
    const Operand xk{x, uint64_t(m), uint64_t(n), L.ldx, false};   // rows of X along K
    const Operand xm{x, uint64_t(m), uint64_t(n), L.ldx, true};
    const Operand ak{Am, d, d, L.ldd, false}, bk{Bm, d, d, L.ldd, false};
    Params p = base;
    p.mode = kGram;
    p.M = p.N = int(d);
    p.out = Am;
    p.ld_out = L.ldd;
    p.batch_out = int64_t(d) * L.ldd;
    p.first = i == 0;
    p.f = float(exp2(double(ea[i] - 2 * ex[i])));
    rc = wide ? product(xk, xk, uint64_t(batch), uint64_t(n), p, dev, width, s)
              : product(xm, xm, uint64_t(batch), uint64_t(m), p, dev, width, s);
    if (rc != SWZ_OK) return rc;

    p = base;
    p.debug_flags = 0;
    p.mode = kPoly;
    p.M = p.N = int(d);
    p.in = Am;
    p.ld_in = L.ldd;
    p.batch_in = int64_t(d) * L.ldd;
    p.out = Bm;
    p.ld_out = L.ldd;
    p.batch_out = int64_t(d) * L.ldd;
    p.u = float(b * exp2(double(eb[i] - ea[i])));
    p.a = float(a);
    p.lost_scale = float(exp2(-double(eb[i])));
    p.f = float(c * exp2(double(eb[i] - 2 * ea[i])));
    rc = product(ak, ak, uint64_t(batch), d, p, dev, width, s);
    if (rc != SWZ_OK) return rc;

    p = base;
    p.debug_flags = 0;
    p.mode = kUpdate;
    p.M = m;
    p.N = n;
    p.first = i == 0;
    p.u = float(exp2(-double(ex[i])));
    p.f = float(exp2(double(-eb[i] - ex[i])));
    p.source = i == 0 ? kFromG : i < masters ? kFromF32 : kFromF16;
    p.in = x;
    p.ld_in = L.ldx;
    p.batch_in = int64_t(m) * L.ldx;
    p.master_in = master;
    if (i == steps - 1) {
      p.y = static_cast<uint8_t*>(Y);
      p.ld_y = m > 1 ? ldy : n;
      p.batch_y = batch > 1 ? batch_stride_y : 0;
      p.y_dtype = y_dtype;
      p.y_wide = ya % 16 == 0 && (m == 1 || (p.ld_y * ys) % 16 == 0) &&
                 (batch == 1 || (p.batch_y * ys) % 16 == 0);
      p.y_lines = p.y_wide && ya % 32 == 0 && (m == 1 || (p.ld_y * ys) % 32 == 0) &&
                  (batch == 1 || (p.batch_y * ys) % 32 == 0);
    } else {
      p.out = xs[(i + 1) & 1];
      p.ld_out = L.ldx;
      p.batch_out = int64_t(m) * L.ldx;
      p.out_scale = float(exp2(double(ex[i + 1])));
      p.master_out = i + 1 < masters ? master : nullptr;
    }
    rc = wide ? product(bk, xm, uint64_t(batch), d, p, dev, width, s)
              : product(xk, bk, uint64_t(batch), d, p, dev, width, s);
    if (rc != SWZ_OK) return rc;
  }
  return SWZ_OK;
}
