// pipe.cuh -- what the 8-bit GEMM and the orthogonalisation share: bounded
// waits on mbarriers, shared-memory matrix descriptors, the tcgen05.mma kinds
// they issue, TMEM loads tied to their wait, and packed fp32 arithmetic.
//
// Every wait is bounded (globaltimer): on expiry the kernel sets the status
// word given by the host, raises the abort flag of its CTA (and of the other
// CTA of a pair) and all roles leave their loops.
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "ptx.cuh"

namespace swz {
namespace pipe {

// Barrier waits and arrivals at CTA scope.  What they order is TMEM and the
// copies' shared memory, which tcgen05's fences and the barriers' own
// transaction counts cover; at cluster scope every arrival is a memory fence
// and every wait drops the L1, which cost a CTA pair that exchanges one tile
// of TMEM per block of K half of its time (8192^3 in 8 bits: 1018 to 494 us).
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

struct Ctl {
  unsigned int* status;      // device status word
  volatile int* abort_flag;  // this CTA's, in shared memory
  uint32_t peer_abort;       // shared::cluster address of the pair's other flag, 0: none
  uint64_t timeout_ns;
};

__device__ __forceinline__ void raise_abort(const Ctl& c) {
  atomicCAS(c.status, 0u, 1u);
  *c.abort_flag = 1;
  if (c.peer_abort)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(c.peer_abort), "r"(1) : "memory");
}

// Waits for the phase of `bar` with parity `parity`; false if the kernel is
// aborting or the bound expired (then the abort is raised).  The timer is not
// read until the hardware's own suspended tries have failed 64 times.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Ctl& c) {
  if (test_wait(bar, parity)) return true;
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1;; ++n) {
    if (try_wait(bar, parity)) return true;
    if ((n & 63u) == 0) {
      if (*c.abort_flag) return false;
      const uint64_t t = ptx::global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > c.timeout_ns) {
        raise_abort(c);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void spin_ns(uint64_t ns) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (ptx::global_timer_ns() - t0 < ns) __nanosleep(1000);
}

// Shared-memory matrix descriptor with the 128-byte swizzle: start address,
// leading and stride byte offsets in 16-byte units, the fixed 0b001 at bits
// 46-48, layout type 2 at bits 61-63.
__device__ __forceinline__ uint64_t sdesc128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((sbo >> 4) & 0x3FFFu) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: D fp32 (bits 4-5 = 1), operand formats at bits 7-9
// and 10-12 (kind::f8f6f4: 0 e4m3, 1 e5m2; kind::f16: 0 fp16), MN-major
// operands at bits 15 (A) and 16 (B), N >> 3 at 17-22, M >> 4 at 24-28.
__host__ __device__ constexpr uint32_t idesc(int a_fmt, int b_fmt, bool a_mn, bool b_mn, int m,
                                             int n) {
  return (1u << 4) | (uint32_t(a_fmt) << 7) | (uint32_t(b_fmt) << 10) |
         (uint32_t(a_mn ? 1 : 0) << 15) | (uint32_t(b_mn ? 1 : 0) << 16) |
         (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// D[tmem] (+)= A * B of 8-bit operands, K = 32 per instruction, fp32 sums.
template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 consecutive 32-bit TMEM columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Waits for this thread's TMEM loads.  The loaded registers pass through the
// statement, so that no use of them can be scheduled before it.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

// Two fp32 values in a 64-bit register, multiplied and added in one
// instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Asynchronous copy of one float to shared memory, zero when !in (`any`: a
// valid address, not read then); copies_arrive arrives on `bar` (one of 32
// lanes) when this thread's copies so far have landed.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool in, const float* any) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(in ? src : any),
               "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float ld_shared(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void ld_shared4(uint32_t addr, float (&v)[4]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(addr)
               : "memory");
}

// 32 x 32 values of a warp, lane i with row i, to lane i with column i.
__device__ __forceinline__ void transpose32(float (&v)[32], uint32_t lane) {
#pragma unroll
  for (uint32_t s = 16; s > 0; s /= 2) {
    const bool high = (lane & s) != 0;
#pragma unroll
    for (uint32_t i = 0; i < 32; ++i) {
      if (i & s) continue;
      const float got = __shfl_xor_sync(0xFFFFFFFFu, high ? v[i] : v[i | s], s);
      if (high) v[i] = got;
      else v[i | s] = got;
    }
  }
}

// Rows of 128 bytes held a row a lane (four pieces of 32 bytes, v[8 c ..] the
// c-th), to and from the order in which a warp stores and loads them: lane l
// then has piece l mod 4 of the rows 4 (l / 4) + j, v[8 j ..] the j-th.  An
// access of the warp is 8 whole lines instead of a quarter of 32, which costs
// the load-store unit a quarter of the time.  Its own inverse.
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[32], uint32_t lane) {
#pragma unroll
  for (uint32_t s = 2; s > 0; s /= 2) {
    const bool high = (lane & s) != 0;
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) {
      if (c & s) continue;
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        uint32_t &a = v[8 * c + k], &b = v[8 * (c | s) + k];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, high ? a : b, s);
        if (high) a = got;
        else b = got;
      }
    }
  }
}

// Eight words from a 16-byte aligned global address.
__device__ __forceinline__ void ld_global_8(const void* p, uint32_t* v) {
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// 32 bytes to a 32-byte aligned global address in one instruction.
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

}  // namespace pipe
}  // namespace swz
