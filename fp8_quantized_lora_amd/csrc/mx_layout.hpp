// Where the exponent bytes of FP4 operands lie.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace falq {

// Exponent bytes of FP4 operands, as the product reads them: [steps x rows16 x 8],
// a step of 256 elements (128 bytes of codes) having eight blocks.  Which chunks of a
// step a lane holds is free, so their bytes lie side by side for both shapes of the
// matrix core's products: a lane group of 16 x 16 x 128 takes blocks g and g + 4, two
// bytes; one of 32 x 32 x 64 takes two of these pairs, four bytes.  Bytes of blocks
// past the row and of rows past the last are 127.
constexpr int kMxStep = 256;
__host__ __device__ constexpr int64_t mx_rows16(int64_t rows) { return (rows + 15) / 16 * 16; }
__host__ __device__ constexpr int64_t mx_steps(int64_t K) { return (K + kMxStep - 1) / kMxStep; }
// the place of block b of a step, and the block at a place
__host__ __device__ constexpr int mx_place_of(int b) { return 2 * (b & 3) + b / 4; }
__host__ __device__ constexpr int mx_block_at(int place) { return place / 2 + 4 * (place & 1); }
__host__ __device__ constexpr int64_t mx_scale_at(int64_t row, int64_t block, int64_t rows16) {
  return ((block >> 3) * rows16 + row) * 8 + mx_place_of((int)(block & 7));
}

}  // namespace falq
