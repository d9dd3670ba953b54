// ops.h -- host-side helpers of the linear-layer operators: their status word
// and tensor maps.
#pragma once
#include <cuda.h>
#include <stdint.h>

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
// elements), boxes of box_cols (64 or fewer) x box_rows of one matrix; swizzle
// of 128 bytes or none.
int encode_half(CUtensorMap* map, const void* base, uint64_t batch, uint64_t rows, uint64_t cols,
                uint64_t ld, uint64_t batch_stride, uint32_t box_cols, uint32_t box_rows,
                bool swizzle);

}  // namespace swz
