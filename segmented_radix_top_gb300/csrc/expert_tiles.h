// Where the tiles of the experts' products lie: whole numbers only, for the
// kernels and, in the instrumented build, for host tests of the largest sizes.
//
// Sizes are below 2^31 - 256 (the limit for rows), so that one tile of 256 more
// still is a 32-bit number; nothing larger is added to them in 32 bits.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace segtopk {

constexpr int kTileQ = 256; // values of q of a tile at most: half of TMEM's columns
constexpr int kStepQ = 32;  // of a tile's width: 16 for each block of a pair

__host__ __device__ __forceinline__ int pieces(int n, int size) { return (n + size - 1) / size; } // size <= 256

// a / b, rounded down, for a >= 0 and b > 0: by a product in 32 bits, which is
// at most one off where the quotient is below 2^22, and a step.
__host__ __device__ __forceinline__ int divide(int a, int b)
{
  if (a >= 1 << 22)
    return a / b;
#ifdef __CUDA_ARCH__
  const float inverse = __frcp_rn((float)b);
#else
  const float inverse = 1.0f / (float)b;
#endif
  int q = (int)((float)a * inverse);
  const int rest = a - q * b;
  q += rest >= b ? 1 : rest < 0 ? -1 : 0;
  return q;
}
// Rounded up, for a > 0. (a + b - 1 would pass 2^31 for the largest a.)
__host__ __device__ __forceinline__ int divide_up(int a, int b) { return divide(a - 1, b) + 1; }

// Part `at` of n > 0 values that go to `parts` = pieces(n, kTileQ) tiles, of
// even widths in steps of kStepQ; none is empty, since all but the last are no
// wider than kTileQ.
struct TilePart {
  int first, width;
};
__host__ __device__ __forceinline__ TilePart even_part(int n, int parts, int at)
{
  const int step = pieces(divide_up(n, parts), kStepQ) * kStepQ;
  const int first = at * step;
  return {first, step < n - first ? step : n - first};
}

// Row i of those that no expert has: the ones before `first`, then those from
// `end` on. In 64 bits: the GPU's warps take a number each to begin with, there
// being that many such rows or not, so end + i may pass 2^31.
__host__ __device__ __forceinline__ int64_t free_row(int first, int end, int64_t i)
{
  return i < first ? i : end + (i - first);
}

} // namespace segtopk
