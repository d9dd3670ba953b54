// int8.h -- what the parts of the 8-bit integer product share on the host side.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace swz {
namespace i8 {

// Longest K: 131071 products of magnitude 2^14 or less stay below 2^31.
constexpr int kMaxK = 131071;

// Rows of x to whole numbers -127 .. 127 and a scale each (arguments checked by the
// caller): as bytes, or as fp16 numbers of the same values (ldq in bytes; whole
// chunks of eight values are written).
int quantize_rows(const void* x, int dtype, int64_t ldx, int M, int K, void* q, int64_t ldq,
                  float* scales, bool half, cudaStream_t s);

}  // namespace i8
}  // namespace swz
