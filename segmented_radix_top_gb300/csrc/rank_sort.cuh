// Stable counting sort of items by a digit of their keys, the step that both
// the sort of token slots by expert (one pass, the key is the digit) and the
// radix sort of token ids (several passes) consist of. Every item's place is
//
//   place(i) = items with a smaller digit
//            + items of the same digit in earlier tiles of the input
//            + items of the same digit before i in its tile,
//
// so equal digits keep their order and the result does not depend on how
// blocks are scheduled. There are two forms:
//
// cluster_sort_kernel, up to kClusterItems items: one launch for all passes.
// 16384 token ids by two digits of 8 bits take 9.7 us, 16384 slots by one
// digit 5.0; the other form's launches 14 and 7.2. Beyond that the eight SMs
// of a cluster are too few (65536 slots: 12.6 us against 6.7).
// A cluster of up to eight blocks holds the items in registers; a pass counts
// digits in shared memory, exchanges the blocks' counts through distributed
// shared memory and, unless it is the last, sends every item to the shared
// memory of the block whose tile its place falls into. Bound by the latency
// of its steps (two cluster barriers and about 30 dependent shared-memory
// accesses a pass) and by the exchange's 8-byte stores, not by the few hundred
// kilobytes it moves.
//
// count_kernel and rank_kernel, any number: two launches a pass over global
// memory, one tile a block; bound by their launches and the latency of a few
// dependent accesses each.
#pragma once

#include <mutex>

#include "common.cuh"
#include "device_prep.h"
#include "rows.cuh"

namespace segtopk {
namespace rows {

struct Digit {
  int shift;
  uint32_t mask;
  __device__ __forceinline__ uint32_t of(uint32_t key) const { return (key >> shift) & mask; }
};

// Items in memory: the key in the low word, its place in the input in the
// high one, so that an item is moved by one access.
__device__ __forceinline__ uint64_t pack(uint32_t key, uint32_t at) { return (uint64_t)at << 32 | key; }

// Exclusive sum over the digits: x is the caller's value for its digit, one
// digit a thread; `all` becomes the sum of all. Two block barriers.
template <int WARPS>
__device__ __forceinline__ uint32_t block_exclusive_sum(uint32_t x, uint32_t* warp_sums, uint32_t* all)
{
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sum = warp_inclusive_sum(x);
  if (lane == 31)
    warp_sums[warp] = sum;
  __syncthreads();
  uint32_t earlier = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    earlier += w < warp ? warp_sums[w] : 0;
    total += warp_sums[w];
  }
  __syncthreads();
  *all = total;
  return earlier + sum - x;
}

// The place of this lane's item among its warp's items of the digit, after
// `seen[digit]` earlier ones, which is brought up to date. Lanes without an
// item (some == false) take part. The lanes are in the items' order; `who`
// (zeros, and zeros again on return) collects the lanes of each digit with
// shared-memory ORs: 7 cycles of an SM per 32 items, where match.any takes
// 55 and a ballot for each of eight digit bits 20.
__device__ __forceinline__ uint32_t place_in_warp(uint32_t* seen, uint32_t* who, uint32_t digit, bool some)
{
  const uint32_t lane = lane_id();
  if (some)
    atomicOr(&who[digit], 1u << lane);
  __syncwarp();
  const uint32_t same = some ? who[digit] : 0, before = some ? seen[digit] : 0;
  const uint32_t ahead = __popc(same & ((1u << lane) - 1));
  __syncwarp();
  if (some && ahead == 0) {
    seen[digit] = before + __popc(same);
    who[digit] = 0;
  }
  __syncwarp();
  return before + ahead;
}

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;

// The warps' counts of a digit (`bins` apart) become the counts of the warps
// before each; returns their sum. All are read before any is written, so
// that the reads do not wait for one another.
__device__ __forceinline__ uint32_t sum_of_warps(uint32_t* counts, int bins, int warps)
{
  uint32_t c[kSortWarps], total = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w)
    c[w] = w < warps ? counts[w * bins] : 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    if (w < warps)
      counts[w * bins] = total;
    total += c[w];
  }
  return total;
}

// Raises a kernel's dynamic shared memory on the current device as far as
// needed; `prep` is the kernel's own.
template <class K>
cudaError_t allow_smem(DevicePrep& prep, K kernel, size_t smem)
{
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess)
    return e;
  if (!DevicePrep::valid(dev))
    return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(prep.mu);
  if (prep.stream_needs(dev, (uint32_t)smem, 1) & DevicePrep::kRaiseSmem) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
      prep.stream_done(dev, (uint32_t)smem, DevicePrep::kRaiseSmem);
  }
  return e;
}

// ---------------------------------------------------------------------------
// One cluster
// ---------------------------------------------------------------------------
constexpr uint32_t kMaxCluster = 8;
constexpr int kMaxRounds = 4; // items of a thread
constexpr uint32_t kBlockItems = kMaxRounds * kSortThreads;
constexpr uint32_t kClusterItems = kMaxCluster * kBlockItems;

// Src: uint32_t key(i) and at(i) of item i. Sink: put(key, at, place) and, in
// a sort of one pass, start(d, first place of digit d).
template <class Src, class Sink>
__global__ void __launch_bounds__(kSortThreads, 1)
cluster_sort_kernel(Src src, Sink sink, uint32_t n, int round_bits, int passes, int digit_bits, int bins)
{
  const uint32_t rounds = 1u << round_bits;
  extern __shared__ uint32_t sh[];
  const uint32_t blocks = cluster_nctarank(), block = cluster_ctarank();
  uint32_t* seen = sh;                        // [warps][bins]
  uint32_t* who = seen + kSortWarps * bins;   // [warps][bins]
  uint32_t* table = who + kSortWarps * bins;  // [blocks][bins], filled by the blocks of the cluster
  uint64_t* items = reinterpret_cast<uint64_t*>(table + (blocks * bins + 1) / 2 * 2); // [tile] at:key, likewise
  const uint32_t tile = rounds * kSortThreads;
  __shared__ uint32_t warp_sums[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t here = warp * rounds * 32 + lane; // in the tile, of round 0
  // items of this thread: those of rounds r with r * 32 < left; warps with any
  const uint32_t left = n - min(n, block * tile + here);
  const int warps = (int)min((uint32_t)kSortWarps, (n - min(n, block * tile) + rounds * 32 - 1) / (rounds * 32));
  if (blocks > 1)
    cluster_arrive(); // every block has to run before its shared memory is written to
  for (int d = threadIdx.x; d < warps * bins; d += kSortThreads)
    seen[d] = who[d] = 0;
  wait_for_previous();
  allow_next(); // here, not later: see the sort's use beside a kernel that clears memory

  uint32_t key[kMaxRounds], at[kMaxRounds], place[kMaxRounds];
#pragma unroll
  for (int r = 0; r < kMaxRounds; ++r) {
    const uint32_t i = block * tile + here + r * 32;
    if ((uint32_t)r < rounds && i < n) {
      key[r] = src.key(i);
      at[r] = src.at(i);
    }
  }
  __syncthreads();
  for (int pass = 0; pass < passes; ++pass) {
    const Digit digit = {pass * digit_bits, passes == 1 ? ~0u : (1u << digit_bits) - 1};
    // places among the warp's items, and the warp's counts
    if (warp < warps)
#pragma unroll
      for (int r = 0; r < kMaxRounds; ++r)
        if ((uint32_t)r < rounds) {
          const bool some = r * 32u < left;
          place[r] = place_in_warp(seen + warp * bins, who + warp * bins, some ? digit.of(key[r]) : 0, some);
        }
    __syncthreads();
    if (blocks > 1 && pass == 0)
      cluster_wait();
    // the warps' counts become the items of the digit in earlier warps
    for (int d = threadIdx.x; d < bins; d += kSortThreads) {
      const uint32_t total = sum_of_warps(seen + d, bins, warps);
      for (uint32_t b = 0; b < blocks; ++b)
        dsmem_st(dsmem_map(smem_addr(table + block * bins + d), b), total);
    }
    __syncwarp(); // cluster barriers want whole warps
    if (blocks > 1)
      cluster_sync();
    else
      __syncthreads();
    // and the first place of the block's items of the digit, kept in who[d]
    uint32_t carried = 0;
    for (int d0 = 0; d0 < bins; d0 += kSortThreads) {
      const int d = d0 + threadIdx.x;
      uint32_t total = 0, before = 0, all;
      if (d < bins)
        for (uint32_t b = 0; b < blocks; ++b) {
          const uint32_t c = table[b * bins + d];
          before += b < block ? c : 0;
          total += c;
        }
      const uint32_t first = carried + block_exclusive_sum<kSortWarps>(total, warp_sums, &all);
      if (d < bins) {
        who[d] = first + before;
        if (block == 0 && passes == 1)
          sink.start(d, first);
      }
      carried += all;
    }
    __syncthreads();
    const bool last = pass + 1 == passes;
#pragma unroll
    for (int r = 0; r < kMaxRounds; ++r) {
      if ((uint32_t)r >= rounds || r * 32u >= left)
        break;
      const uint32_t d = digit.of(key[r]);
      const uint32_t p = who[d] + seen[warp * bins + d] + place[r];
      if (last) {
        sink.put(key[r], at[r], p);
      } else {
        dsmem_st(dsmem_map(smem_addr(items + (p & (tile - 1))), p / kSortThreads >> round_bits),
                 pack(key[r], at[r]));
      }
    }
    if (last)
      break; // nothing is written to another block's memory after the barrier above
    __syncwarp();
    if (blocks > 1)
      cluster_sync();
    else
      __syncthreads();
#pragma unroll
    for (int r = 0; r < kMaxRounds; ++r)
      if ((uint32_t)r < rounds && r * 32u < left) {
        const uint64_t item = items[here + r * 32];
        key[r] = (uint32_t)item;
        at[r] = (uint32_t)(item >> 32);
      }
    for (int d = threadIdx.x; d < warps * bins; d += kSortThreads)
      seen[d] = who[d] = 0;
    __syncthreads();
  }
}

template <class Src, class Sink>
cudaError_t launch_cluster_sort(Src src, Sink sink, uint32_t n, int passes, int digit_bits, int bins,
                                uint32_t blocks, cudaStream_t stream)
{
  auto kernel = cluster_sort_kernel<Src, Sink>;
  int round_bits = 0; // a power of two, so that a place's block and slot are bits of it
  while (blocks * kSortThreads << round_bits < n)
    ++round_bits;
  const size_t tile = passes > 1 ? (size_t)kSortThreads << round_bits : 0;
  const size_t smem = ((2 * kSortWarps + blocks) * (size_t)bins + 1 + 2 * tile) * 4;
  static DevicePrep prep;
  const cudaError_t e = allow_smem(prep, kernel, smem);
  if (e != cudaSuccess)
    return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, src, sink, n, round_bits, passes, digit_bits, bins);
}

// ---------------------------------------------------------------------------
// Any number of blocks
// ---------------------------------------------------------------------------
constexpr uint32_t kTile = 2048; // items of a tile (more where kMaxTiles tiles do not cover them)
constexpr uint32_t kMaxTiles = 128;

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

template <class Src>
__global__ void __launch_bounds__(512)
count_kernel(Src src, Digit digit, uint32_t n, uint32_t tile, int bins, uint32_t* counts)
{
  extern __shared__ uint32_t sh[];
  for (int d = threadIdx.x; d < bins; d += 512)
    sh[d] = 0;
  __syncthreads();
  wait_for_previous();
  const uint32_t lo = blockIdx.x * tile, hi = min(n, lo + tile);
  for (uint32_t i = lo + threadIdx.x; i < hi; i += 512)
    atomicAdd(&sh[digit.of(src.key(i))], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += 512)
    counts[(size_t)blockIdx.x * bins + d] = sh[d];
}

template <class Src, class Sink>
__global__ void __launch_bounds__(kSortThreads)
rank_kernel(Src src, Digit digit, Sink sink, uint32_t n, uint32_t tile, int bins, const uint32_t* counts, bool only)
{
  extern __shared__ uint32_t sh[];
  uint32_t* seen = sh;                      // [warps][bins]
  uint32_t* who = sh + kSortWarps * bins;   // [warps][bins]
  uint32_t* base = who + kSortWarps * bins; // [bins]
  __shared__ uint32_t warp_sums[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int d = threadIdx.x; d < kSortWarps * bins; d += kSortThreads)
    seen[d] = who[d] = 0;
  __syncthreads();
  wait_for_previous();
  // each warp counts its own share of the tile
  const uint32_t share = tile / kSortWarps; // a multiple of 32
  const uint32_t lo = min(n, blockIdx.x * tile + warp * share), hi = min(n, lo + share);
  for (uint32_t i = lo + lane; i < hi; i += 32)
    atomicAdd(&seen[warp * bins + digit.of(src.key(i))], 1u);
  __syncthreads();
  // per digit: the warps' counts become their first places within the tile;
  // the items of the digit in all tiles and in the tiles before this one
  uint32_t carried = 0;
  for (int d0 = 0; d0 < bins; d0 += kSortThreads) {
    const int d = d0 + threadIdx.x;
    uint32_t total = 0, before = 0, all;
    if (d < bins) {
      sum_of_warps(seen + d, bins, kSortWarps);
#pragma unroll 16
      for (uint32_t b = 0; b < gridDim.x; ++b) {
        const uint32_t c = counts[(size_t)b * bins + d];
        before += b < blockIdx.x ? c : 0;
        total += c;
      }
    }
    const uint32_t first = carried + block_exclusive_sum<kSortWarps>(total, warp_sums, &all);
    if (d < bins) {
      base[d] = first + before;
      if (blockIdx.x == 0 && only)
        sink.start(d, first);
    }
    carried += all;
  }
  __syncthreads();
  allow_next();
#pragma unroll 2
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t i = i0 + lane;
    const bool some = i < hi;
    const uint32_t key = some ? src.key(i) : 0, d = some ? digit.of(key) : 0;
    const uint32_t in_tile = place_in_warp(seen + warp * bins, who + warp * bins, d, some);
    if (some)
      sink.put(key, src.at(i), base[d] + in_tile);
  }
}

template <class Src, class Sink>
cudaError_t launch_rank(Src src, Digit digit, Sink sink, uint32_t n, Tiling t, int bins, const uint32_t* counts,
                        bool only, cudaStream_t stream)
{
  auto kernel = rank_kernel<Src, Sink>;
  const size_t smem = (size_t)bins * 4 * (2 * kSortWarps + 1);
  static DevicePrep prep;
  const cudaError_t e = allow_smem(prep, kernel, smem);
  return e != cudaSuccess ? e : launch(kernel, dim3(t.tiles), kSortThreads, smem, stream, src, digit, sink, n, t.items,
                                       bins, counts, only);
}

struct ItemSource {
  const uint64_t* items;
  __device__ __forceinline__ uint32_t key(uint32_t i) const { return (uint32_t)items[i]; }
  __device__ __forceinline__ uint32_t at(uint32_t i) const { return (uint32_t)(items[i] >> 32); }
};
struct ItemSink {
  uint64_t* items;
  __device__ __forceinline__ void put(uint32_t key, uint32_t at, uint32_t place) const { items[place] = pack(key, at); }
  __device__ __forceinline__ void start(int, uint32_t) const {}
};

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// A sort of n keys by their lowest passes * digit_bits bits; with one pass,
// keys are below `bins`.
struct SortPlan {
  uint32_t n;
  int passes, digit_bits, bins;
  Tiling tiles; // items 0: one cluster
  size_t copy() const { return tiles.items && passes > 1 ? (size_t)n * 8 : 0; } // bytes of a copy of all items
  size_t counts() const { return tiles.items ? (size_t)tiles.tiles * (size_t)bins * 4 : 0; }
};
inline SortPlan sort_plan(int64_t n, int passes, int digit_bits, int bins)
{
  return {(uint32_t)n, passes, digit_bits, bins, n > (int64_t)kClusterItems ? tiling(n) : Tiling{0, 0}};
}

// `copies`: two copies of the items (plan.copy() bytes each) for passes that
// are not the last; counts: plan.counts() bytes. ONE_PASS: plan.passes is 1.
// Returns the number of launches, or -1 with *e set.
template <bool ONE_PASS, class Src, class Sink>
int sort(const SortPlan& p, Src src, Sink sink, uint64_t* const (&copies)[2], uint32_t* counts, cudaStream_t stream,
         cudaError_t* e)
{
  if (!p.tiles.items) {
    uint32_t blocks = 1;
    while (blocks * kBlockItems < p.n)
      blocks *= 2;
    *e = launch_cluster_sort(src, sink, p.n, p.passes, p.digit_bits, p.bins, blocks, stream);
    return *e == cudaSuccess ? 1 : -1;
  }
  auto pass = [&](auto from, auto to, int k) {
    const Digit digit = {k * p.digit_bits, p.passes == 1 ? ~0u : (1u << p.digit_bits) - 1};
    *e = launch(count_kernel<decltype(from)>, dim3(p.tiles.tiles), 512, (size_t)p.bins * 4, stream, from, digit, p.n,
                p.tiles.items, p.bins, counts);
    if (*e != cudaSuccess)
      return;
    *e = launch_rank(from, digit, to, p.n, p.tiles, p.bins, counts, p.passes == 1, stream);
  };
  auto from = [&](int k) { return ItemSource{copies[k & 1]}; };
  auto to = [&](int k) { return ItemSink{copies[k & 1]}; };
  *e = cudaSuccess;
  if constexpr (ONE_PASS) {
    pass(src, sink, 0);
  } else {
    for (int k = 0; k < p.passes && *e == cudaSuccess; ++k) {
      const bool last = k + 1 == p.passes;
      if (k == 0)
        last ? pass(src, sink, k) : pass(src, to(0), k);
      else
        last ? pass(from(k - 1), sink, k) : pass(from(k - 1), to(k), k);
    }
  }
  return *e == cudaSuccess ? 2 * p.passes : -1;
}

} // namespace rows
} // namespace segtopk
