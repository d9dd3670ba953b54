// linear_fp8.cu -- y = x W^T with W kept in 8 bits: x (M x K; fp16, bf16 or
// fp32) is quantised in row blocks (e4m3) into the caller's workspace and
// multiplied as swz_gemm_fp8 does.  The product of few rows starts reading W
// while the quantiser runs.  (One kernel for both was tried for up to 16 rows:
// mma.sync on W streamed through registers, x brought to 8 bits by every CTA.
// 10.7 us for one row of 4096 x 4096 against 8.1: the 8-bit form of mma.sync is
// converted to 16 bits on the way, and each CTA pays the quantisation.)
#include "common.h"
#include "ops.h"

namespace swz {
namespace f8 {

// workspace: 8-bit x with rows of a multiple of 16 bytes, then its scales
static void workspace_split(int M, int K, int64_t* ldq, uint64_t* q_bytes, uint64_t* total) {
  *ldq = (int64_t(K) + 15) / 16 * 16;
  *q_bytes = (uint64_t(M) * uint64_t(*ldq) + 255u) & ~uint64_t(255);
  *total = *q_bytes + (uint64_t(K) + 127) / 128 * uint64_t(M) * 4;
}

}  // namespace f8
}  // namespace swz

using namespace swz;

extern "C" int swz_linear_fp8_workspace_size(int M, int N, int K, uint64_t* h_bytes) {
  if (!h_bytes || M < 0 || N < 0 || K < 0) return SWZ_EINVAL;
  *h_bytes = 0;
  if (M == 0 || N == 0 || K == 0) return SWZ_OK;
  int64_t ldq;
  uint64_t q_bytes;
  f8::workspace_split(M, K, &ldq, &q_bytes, h_bytes);
  return SWZ_OK;
}

extern "C" int swz_linear_fp8(const void* x, int dtype, int64_t ldx, const swz_fp8_matrix* W,
                              void* y, int64_t ldy, int y_dtype, int M, int N, int K,
                              void* d_workspace, uint64_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !W) return SWZ_EINVAL;
  for (int d : {dtype, y_dtype})
    if (d != SWZ_F16 && d != SWZ_BF16 && d != SWZ_F32) return SWZ_EINVAL;
  if (W->fmt != SWZ_E4M3 && W->fmt != SWZ_E5M2) return SWZ_EINVAL;
  if (W->block != SWZ_BLOCK_ROW && W->block != SWZ_BLOCK_SQUARE) return SWZ_EINVAL;
  if (M == 0 || N == 0) return SWZ_OK;
  const int64_t es = dtype == SWZ_F32 ? 4 : 2, ys = y_dtype == SWZ_F32 ? 4 : 2;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x);
  if (!y || reinterpret_cast<uintptr_t>(y) % uintptr_t(ys) != 0 || (M > 1 && ldy < N))
    return SWZ_EINVAL;
  const int64_t kb = (int64_t(K) + 127) / 128;
  if (K > 0 && (!x || xa % uintptr_t(es) != 0 || (M > 1 && ldx < K) || !W->data ||
                !aligned16(W->data) || W->ld < K || W->ld % 16 != 0 || !W->scales ||
                !aligned4(W->scales) ||
                W->ld_scales < (W->block == SWZ_BLOCK_SQUARE ? kb : int64_t(N))))
    return SWZ_EINVAL;
  int64_t ldq;
  uint64_t q_bytes, total;
  f8::workspace_split(M, K, &ldq, &q_bytes, &total);
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  if (K > 0 && (!ws || !aligned16(ws) || workspace_bytes < total)) return SWZ_EINVAL;
  DeviceInfo dev{};
  const int rc = current_device(&dev);
  if (rc != SWZ_OK) return rc;
  swz_fp8_matrix a = {};
  a.data = ws;
  a.ld = ldq;
  a.scales = reinterpret_cast<float*>(ws + q_bytes);
  a.ld_scales = M;
  a.fmt = SWZ_E4M3;
  a.block = SWZ_BLOCK_ROW;
  if (K > 0) {
    const int rq = swz_quantize_fp8(x, dtype, ldx, M, K, SWZ_BLOCK_ROW, SWZ_E4M3, ws, ldq,
                                    reinterpret_cast<float*>(ws + q_bytes), M, nullptr, 0, nullptr,
                                    0, stream);
    if (rq != SWZ_OK) return rq;
  }
  return gemm_fp8(&a, W, y, ldy, y_dtype, M, N, K, nullptr, stream, /*early_b=*/true);
}
