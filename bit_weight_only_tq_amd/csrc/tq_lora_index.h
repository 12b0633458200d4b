// Where the adapters' kernel (lora.hip) reads B: plain integers, also compiled on
// the host, where a test walks a whole call's reads.
//
// A buffer descriptor checks the offset of a lane against the buffer's end.  The
// scalar offset of the instruction is no part of that check for the compiler, so
// whatever may lie past the end has to be in the lane's own offset.
#pragma once

#include <stdint.h>

#if !defined(__HIPCC__)
#define __host__
#define __device__
#endif

namespace tq {

// Lies past the end of any buffer (of fewer than 2^31 bytes).
constexpr uint32_t kNowhere = 0x80000000u;

// First of the 32 columns of step i of a wave, of W waves, in a chunk of `cols`
// columns that begins at n_lo.  Two steps in a row where there are enough columns
// for every wave, so that a wave's stores fill the cache lines that they begin.
__host__ __device__ constexpr int lora_step(int n_lo, int cols, int W, int wave, int i) {
    return cols >= 64 * W ? n_lo + 64 * wave + 32 * (i & 1) + (i >> 1) * (64 * W) : n_lo + 32 * wave + i * (32 * W);
}

// Byte offset, from an adapter's first value of B [N, r], of the eight values that lane
// 16 g + i16 takes for tile t and ranks 32 st on, columns n .. n + 31: matrix row
// 4 g' + e of tile t is column n + 8 g' + 4 t + e, so that a lane ends with 8 columns
// in a row of one row.  `lane` is the part that no step changes, `step` the columns'.
// Rows of B past the last lie past its end, ranks past r nowhere, and neither comes
// back by the sum: `step` is at most (2^22 + 2^9) r values, of a matrix of 2^29 at most.
__host__ __device__ constexpr uint32_t lora_b_lane(int r, int i16, int g, int t, int st) {
    return 32 * st + 8 * g < r ? ((uint32_t)(8 * (i16 >> 2) + 4 * t + (i16 & 3)) * (uint32_t)r + 8u * g + 32u * st) * 2u : kNowhere;
}
__host__ __device__ constexpr uint32_t lora_b_step(int r, int n) { return (uint32_t)n * (uint32_t)r * 2u; }

}  // namespace tq
