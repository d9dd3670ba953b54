// ops.h -- host-side helpers of the linear-layer operators: their status word
// and tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "swz.h"

namespace swz {

// Device address of the current device's status word of these operators
// (looked up once per device, outside stream capture).
int op_status_word(unsigned int** word);

// Reads and clears that word of the current device; *expired: a bounded wait
// ran out since the last call.
int take_op_status(bool* expired);

// Tensor map of a row-major rows x cols matrix of bytes with rows ld bytes
// apart, boxes of 128 bytes x box_rows, 128-byte swizzle; reads outside are 0.
int encode_bytes(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld,
                 uint32_t box_rows);

// The same for batch matrices of 16-bit elements (ld and batch stride in
// elements), boxes of box_cols (64 or fewer) x box_rows of one matrix, 128-byte
// swizzle.
int encode_half(CUtensorMap* map, const void* base, uint64_t batch, uint64_t rows, uint64_t cols,
                uint64_t ld, uint64_t batch_stride, uint32_t box_cols, uint32_t box_rows);

// swz_gemm_fp8; `early_b`: the kernel before in the stream is the quantiser of
// A, launched by the same caller, and B may be read while it runs.
int gemm_fp8(const swz_fp8_matrix* A, const swz_fp8_matrix* B, void* C, int64_t ldc, int c_dtype,
             int M, int N, int K, const swz_gemm_fp8_opts* opts, void* stream, bool early_b);

// Its kernel for up to kFewRows rows of A (arguments checked by the caller;
// split 0: automatic).  16 rows, 4096 x 4096: 6.9 us against 9.8 with 128-row
// tiles, 8192 x 8192 14.5 against 17.0; 32 rows 7.7 against 9.5 and 14.9
// against 17.1, and of 10240 x 4096 12.3 against 12.4.  The tensor core's N and
// the accumulators end at 32.
constexpr int kFewRows = 32;
int gemm_fp8_rows(const swz_fp8_matrix& A, const swz_fp8_matrix& B, void* C, int64_t ldc,
                  int c_dtype, int M, int N, int K, int split, uint32_t debug_flags,
                  uint64_t timeout_ns, bool early_b, int num_sms, cudaStream_t stream);

}  // namespace swz
