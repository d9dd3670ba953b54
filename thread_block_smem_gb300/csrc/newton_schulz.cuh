// newton_schulz.cuh -- what the two forms of swz_newton_schulz share.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "f8.cuh"
#include "swz.h"

namespace swz {
namespace ns {

// per matrix of the batch: X = G * p1 * p2 * f, and the first fp16 X is G * p1
// * p2; a later fp16 X is X times the step's power of two times `up`, a power
// of two above 1 when |G| is so far below eps that X is tiny (down = 1 / up)
struct Scale {
  float p1, p2, f, up, down;
};

// From the sums of squares of G, of 2^-80 G and of 2^80 G (the one that neither
// overflowed nor underflowed is used) and its number of elements.  `headroom`:
// |G| / (|G| + eps) below this leaves room to scale X up.
__device__ __forceinline__ Scale make_scale(const double (&d)[3], double count, double eps,
                                            double headroom) {
  double norm;
  if (!(d[0] < 1e36)) norm = sqrt(d[1]) * 0x1p80;
  else if (d[0] > 1e-30) norm = sqrt(d[0]);
  else norm = sqrt(d[2]) * 0x1p-80;
  Scale sc;
  // a power of two with norm * 2^e between sqrt(count) / 8 and sqrt(count)
  int e = 0;
  if (norm > 0.0 && norm < 1e300) e = ilogb(count) / 2 - ilogb(norm) - 1;
  const double div = norm + eps;
  sc.p1 = ldexpf(1.f, e / 2);
  sc.p2 = ldexpf(1.f, e - e / 2);
  sc.f = div > 0.0 ? float(ldexp(1.0, -e) / div) : (div == 0.0 ? 0.f : float(div));
  // X grows from |G| / (|G| + eps) by known factors, its bound by others
  int z = 0;
  if (norm > 0.0 && norm < div * headroom) z = ilogb(headroom) + ilogb(div) - ilogb(norm) - 2;
  z = z < 0 ? 0 : z > 100 ? 100 : z;
  sc.up = ldexpf(1.f, z);
  sc.down = ldexpf(1.f, -z);
  return sc;
}

// plain loads, as f8::load8's; p may also be where the result goes
__device__ __forceinline__ float load_any(const uint8_t* p, int64_t at, int dtype) {
  if (dtype == SWZ_F32) return reinterpret_cast<const float*>(p)[at];
  if (dtype == SWZ_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[at]);
  return __half2float(reinterpret_cast<const __half*>(p)[at]);
}
__device__ __forceinline__ void store_any(uint8_t* p, int64_t at, float v, int dtype) {
  if (dtype == SWZ_F32) reinterpret_cast<float*>(p)[at] = v;
  else if (dtype == SWZ_BF16) reinterpret_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  else reinterpret_cast<__half*>(p)[at] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

constexpr int kMaxSteps = 64;
constexpr int kSmallSide = 128, kSmallLong = 2048;  // largest of newton_schulz_small.cu

struct SmallParams {
  const uint8_t* g;
  int64_t ld_g, batch_g;
  int g_dtype;
  uint8_t* y;
  int64_t ld_y, batch_y;
  int y_dtype;
  int wide;     // the short side is the rows of G
  int d, len;   // short and long side
  int steps;
  double eps, headroom;
  uint32_t ranks, cols;  // CTAs of a matrix, long columns of each
  uint32_t debug_flags;
  unsigned int* status;
  uint64_t timeout_ns;
  // by step: A = P * fa, B = ub * A + fb * A A, X = D * k1, the operands hold
  // X * sx and D a X * ad / a of that (all but for the matrix's Scale)
  float fa[kMaxSteps], ub[kMaxSteps], fb[kMaxSteps], k1[kMaxSteps], sx[kMaxSteps], ad[kMaxSteps];
};

int small_pays(int batch, int len, bool* pays);
int launch_small(SmallParams p, int batch, cudaStream_t stream);

}  // namespace ns
}  // namespace swz
