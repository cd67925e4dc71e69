// small_div.cuh -- division of small indexes by a number that a launch fixes.
#pragma once

#include <stdint.h>

namespace msa {

// x / q for 0 <= x < 2^18 and q < 2^14 with m = ceil(2^32 / q): x m / 2^32 exceeds x / q by less
// than 2^18 / 2^32 < 1 / q.  (q = 1 has m = 2^32, which does not fit: m = 0 stands for it.)
__device__ __forceinline__ int small_div(int x, uint32_t m) { return m ? (int)__umulhi((uint32_t)x, m) : x; }
inline uint32_t magic(int q) { return q == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + q - 1) / q); }

}  // namespace msa
