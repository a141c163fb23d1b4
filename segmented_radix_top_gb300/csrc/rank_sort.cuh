// Stable counting sort of items by a digit, the step that both the sort of
// token slots by expert (one pass, digit = expert) and the radix sort of
// token ids (several passes of up to 9 bits) consist of.
//
// The items are cut into `blocks` contiguous tiles. count_kernel writes each
// tile's count of every digit; rank_kernel gives every item its place,
//
//   place(i) = items with a smaller digit
//            + items of the same digit in earlier tiles
//            + items of the same digit before i in its tile,
//
// so equal digits keep their order and the result does not depend on how
// the blocks are scheduled. A single tile needs rank_kernel alone.
#pragma once

#include "rows.cuh"

namespace segtopk {
namespace rows {

constexpr uint32_t kTile = 2048; // items of a tile (more where kMaxTiles tiles do not cover them)
constexpr uint32_t kMaxTiles = 128;
constexpr int kWideBins = 513; // more bins than this take rank_kernel's 8-warp form

struct Tiling {
  uint32_t items, tiles;
};
inline Tiling tiling(int64_t n)
{
  const uint32_t tiles = (uint32_t)std::min<int64_t>(kMaxTiles, std::max<int64_t>(1, (n + kTile - 1) / kTile));
  uint32_t items = (uint32_t)((n + tiles - 1) / tiles);
  items = std::max<uint32_t>((items + 511) / 512 * 512, 512); // whole warps' shares
  return {items, (uint32_t)std::max<int64_t>(1, (n + items - 1) / items)};
}
inline size_t count_bytes(Tiling t, int bins) { return t.tiles > 1 ? (size_t)t.tiles * (size_t)bins * 4 : 0; }

// Src: digit(i) < bins of item i.
template <class Src>
__global__ void __launch_bounds__(512) count_kernel(Src src, uint32_t n, uint32_t tile, int bins, uint32_t* counts)
{
  extern __shared__ uint32_t sh[];
  for (int d = threadIdx.x; d < bins; d += 512)
    sh[d] = 0;
  __syncthreads();
  wait_for_previous();
  const uint32_t lo = blockIdx.x * tile, hi = min(n, lo + tile);
  for (uint32_t i = lo + threadIdx.x; i < hi; i += 512)
    atomicAdd(&sh[src.digit(i)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += 512)
    counts[(size_t)blockIdx.x * bins + d] = sh[d];
}

// Src: also Item load(i) with a member digit. Sink: put(i, item, place) and,
// called by the first block for every digit, start(d, first place of d).
template <int WARPS, class Src, class Sink>
__global__ void __launch_bounds__(WARPS * 32) rank_kernel(Src src, Sink sink, uint32_t n, uint32_t tile, int bins,
                                                          const uint32_t* counts)
{
  constexpr int NT = WARPS * 32;
  extern __shared__ uint32_t sh[];
  uint32_t* base = sh;        // [bins]
  uint32_t* mine = sh + bins; // [WARPS][bins]
  __shared__ uint32_t warp_sum[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int d = threadIdx.x; d < bins * WARPS; d += NT)
    mine[d] = 0;
  __syncthreads();
  wait_for_previous();
  // each warp counts its own share of the tile
  const uint32_t share = tile / WARPS; // a multiple of 32
  const uint32_t lo = min(n, blockIdx.x * tile + warp * share), hi = min(n, lo + share);
  uint32_t* own = mine + warp * bins;
  for (uint32_t i = lo + lane; i < hi; i += 32)
    atomicAdd(&own[src.digit(i)], 1u);
  __syncthreads();
  // per digit: the warps' counts become their first places within the tile;
  // the items of the digit in all tiles and in the tiles before this one
  uint32_t carried = 0;
  for (int d0 = 0; d0 < bins; d0 += NT) {
    const int d = d0 + threadIdx.x;
    uint32_t total = 0, before = 0;
    if (d < bins) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const uint32_t c = mine[w * bins + d];
        mine[w * bins + d] = total;
        total += c;
      }
      if (gridDim.x > 1) {
        total = 0;
#pragma unroll 8
        for (uint32_t b = 0; b < gridDim.x; ++b) {
          const uint32_t c = *(counts + (size_t)b * bins + d);
          before += b < blockIdx.x ? c : 0;
          total += c;
        }
      }
    }
    // exclusive sum of the totals over the digits
    uint32_t sum = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, sum, o);
      if (lane >= o)
        sum += y;
    }
    if (lane == 31)
      warp_sum[warp] = sum;
    __syncthreads();
    uint32_t earlier = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      earlier += w < warp ? warp_sum[w] : 0;
      all += warp_sum[w];
    }
    if (d < bins) {
      const uint32_t first = carried + earlier + sum - total;
      base[d] = first + before;
      if (blockIdx.x == 0)
        sink.start(d, first);
    }
    carried += all;
    __syncthreads(); // warp_sum is written again; base is read below
  }
  allow_next();
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t i = i0 + lane;
    const bool some = i < hi;
    const unsigned on = __ballot_sync(kAll, some);
    if (some) {
      const auto item = src.load(i);
      const unsigned same = __match_any_sync(on, item.digit);
      const uint32_t seen = own[item.digit];
      const uint32_t ahead = __popc(same & ((1u << lane) - 1));
      __syncwarp(on);
      if (ahead == 0)
        own[item.digit] = seen + __popc(same);
      sink.put(i, item, base[item.digit] + seen + ahead);
    }
    __syncwarp();
  }
}

// One stable pass: `counts` holds count_bytes(t, bins) bytes. Returns the
// number of launches, or -1 with *e set.
template <class Src, class Sink>
int rank_pass(Src src, Sink sink, uint32_t n, Tiling t, int bins, uint32_t* counts, cudaStream_t stream, cudaError_t* e)
{
  int launches = 1;
  if (t.tiles > 1) {
    *e = launch(count_kernel<Src>, dim3(t.tiles), 512, (size_t)bins * 4, stream, src, n, t.items, bins, counts);
    if (*e != cudaSuccess)
      return -1;
    ++launches;
  }
  // the warps' counters stay within the 48 KB that need no opt-in
  if (bins <= kWideBins)
    *e = launch(rank_kernel<16, Src, Sink>, dim3(t.tiles), 512, (size_t)bins * 4 * 17, stream, src, sink, n, t.items,
                bins, (const uint32_t*)counts);
  else
    *e = launch(rank_kernel<8, Src, Sink>, dim3(t.tiles), 256, (size_t)bins * 4 * 9, stream, src, sink, n, t.items,
                bins, (const uint32_t*)counts);
  return *e == cudaSuccess ? launches : -1;
}

} // namespace rows
} // namespace segtopk
