// Where the E8M0 scales of MX activations and weights live (used by every
// kernel that writes them).
#pragma once

#include "common.cuh"

namespace w4 {
namespace {

// Byte offset of the scale of (row r, 32-element block kb) in the tensor-core
// layout of a matrix with K columns: 512-byte atoms of 128 rows x 4 blocks,
// row r of an atom at 16 * (r % 32) + 4 * (r / 32), block kb % 4 in the byte
// of that 32-bit word; atoms ordered by k within a 128-row band.
__host__ __device__ __forceinline__ int64_t mma_sf_offset(int64_t r, int64_t kb, int64_t K)
{
    return (((r >> 7) * (K >> 7) + (kb >> 2)) << 9) + ((r & 31) << 4) + (((r >> 5) & 3) << 2) + (kb & 3);
}

}  // namespace
}  // namespace w4
