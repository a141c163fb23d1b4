// Each expert's matrix product of its rows, and its gradients
// (segtopk_expert_matmul, segtopk_expert_matmul_f8 and
// segtopk_expert_matmul_weights in include/segtopk.h).
//
// All are products of tiles D[p, q] = sum_c P[p, c] Q[q, c], 128 values of p
// by up to 256 of q, on the tensor cores (tcgen05, sums in TMEM in 32 bits):
//   forward         p an expert's outputs, q its rows, c the width
//   rows' gradient  p an expert's inputs, q its rows, c the outputs: the
//                   forward product with the weights read the other way round
//   weights'        p and q an expert's inputs and outputs (the dense one of
//                   the weights as p), c its rows
// The weights are p even where there are few rows: a tile is as wide as the
// expert's rows, in steps of 16, so one kernel serves 1 row and 10 000, and a
// lane of the sums is a column of the result, whose 32 neighbours lie side by
// side in memory.
//
// Operands come by TMA in blocks of 128 bytes of c, a ring of four stages of
// 48 KB. Warps have one part each: 0 copies, 1 issues products, 2 and 3 fetch
// scales, 4 to 11 take the sums out of TMEM, which holds two sets of them, so
// that they work while the next set is computed. Blocks stay on their SM and
// take tile after tile; each finds the tiles from the experts' offsets, which
// the host never reads.
//
// 8-bit operands: the sum over one block of 128 values of c has one scale for
// each row and one for the weights' tile, so every block's sums are taken out
// of TMEM, multiplied and added up in registers in 32 bits.
#include <atomic>
#include <cuda.h>

#include "common.cuh"
#include "rows.cuh"

namespace segtopk {
namespace {
using namespace rows;

constexpr int kThreads = 384;
constexpr int kSumWarps = 8;     // of them the last
constexpr int kTileP = 128;      // lanes of TMEM
constexpr int kTileQ = 256;      // half of its columns
constexpr int kStages = 4;
constexpr int kBytesP = kTileP * 128, kBytesQ = kTileQ * 128;
constexpr int kStageBytes = kBytesP + kBytesQ;
constexpr int kBox = 32;         // rows of one copy of an expert's rows
constexpr int kDepth = 64;       // rows of one copy where c runs over rows
constexpr int kMaxExperts = SEGTOPK_MAX_EXPERTS;

enum Kind { kForward8, kForward, kForwardTurned, kWeights };

struct Control {
  uint64_t full[kStages], empty[kStages];       // copies have landed; products have read them
  uint64_t sums_full[2], sums_empty[2];         // TMEM's halves
  uint64_t drained;                             // products behind a wait that ran out
  uint32_t tmem;
  int failed;                                   // a wait ran out: everybody leaves
  int part[kThreads / 32];
  int tile_start[kMaxExperts + 1];              // experts' first tiles
  int row_start[kMaxExperts + 1];               // and rows
};
constexpr size_t kShared = 1024 + (size_t)kStages * kStageBytes + sizeof(Control);
static_assert(kShared <= 227 * 1024, "shared memory of a block");

struct Sizes {
  int64_t num_rows;     // slots; those from the last offset on have no expert
  int experts;
  int p, q, c;          // sizes; an expert's rows take the place of one
  int step;             // kForward8: the tiles' q
  uint32_t instruction; // types and majors of the operands
  int64_t out_stride;   // between rows of the result, which are dense
  bool out_vectors;     // kForward8: they can be written 16 bytes at a time
  const float* row_scales;
  int64_t scale_stride;
  const float* weight_scales;
};

// ---------------------------------------------------------------------------
// Tensor memory and tensor cores
// ---------------------------------------------------------------------------
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tile_load(void* to, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
               "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(to)),
               "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
               : "memory");
}

// Shared-memory operand of 128-byte rows, swizzled over eight of them. Rows
// of c: 8 rows are 1024 bytes. Rows of p or q: 64 of these by 8 of c are 1024
// bytes, the next 8 of c follow, the next 64 are a copy further on.
template <bool ROWS_OF_C>
__device__ __forceinline__ uint64_t operand(uint32_t address)
{
  constexpr uint64_t lead = ROWS_OF_C ? 1 : kDepth * 128 / 16;
  return (uint64_t)(address >> 4) | lead << 16 | (uint64_t)(1024 / 16) << 32 | 1ull << 46 | 2ull << 61;
}

template <bool EIGHT>
__device__ __forceinline__ void multiply(uint32_t sums, uint64_t p, uint64_t q, uint32_t instruction, bool add)
{
  if constexpr (EIGHT)
    asm volatile("{\n .reg .pred a;\n setp.ne.b32 a, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, a;\n}" ::"r"(sums),
                 "l"(p), "l"(q), "r"(instruction), "r"((uint32_t)add)
                 : "memory");
  else
    asm volatile("{\n .reg .pred a;\n setp.ne.b32 a, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, a;\n}" ::"r"(sums),
                 "l"(p), "l"(q), "r"(instruction), "r"((uint32_t)add)
                 : "memory");
}
// Arrives at `bar` once the products issued so far are done.
__device__ __forceinline__ void commit(uint64_t* bar)
{
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar)
{
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Columns of this warp's 32 lanes; the values are there after sums_wait()
// has been given them.
__device__ __forceinline__ void sums_load(uint32_t (&v)[16], uint32_t at)
{
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
               : "r"(at));
}
__device__ __forceinline__ void sums_wait(uint32_t (&v)[16])
{
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void sums_load(uint32_t (&v)[32], uint32_t at)
{
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
               "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                 "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
                 "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
                 "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
               : "r"(at));
}
__device__ __forceinline__ void sums_wait(uint32_t (&v)[32])
{
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

// Waits for the phase of `bar` with this parity; false, for good, after about
// a second, or once another wait of the block has run out.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Control& sh)
{
  if (mbar_try_wait(bar, parity))
    return true;
  const long long start = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*(volatile int*)&sh.failed)
      return false;
    if (clock64() - start > kWaitLimitCycles) {
      *(volatile int*)&sh.failed = 1;
      raise_error(kErrCopyTimeout);
      return false;
    }
  }
  return true;
}

// A place in a ring of N and the parity of the passes over it.
template <int N>
struct Ring {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next()
  {
    if (++at == N) {
      at = 0;
      parity ^= 1;
    }
  }
};

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
__host__ __device__ __forceinline__ int pieces(int n, int size) { return (n + size - 1) / size; }

struct Tile {
  int expert;
  int p;          // first
  int q, width;   // first and how many; rounded up to 16 there are
  int row, rows;  // the expert's rows
  int blocks;     // of c
};

// Tiles of an expert with this many rows. Where q are its rows, or its inputs
// or outputs, it goes to as few tiles as hold it, of even widths in steps of
// 16; none is empty, since all but the last are no wider than kTileQ.
template <Kind K>
__device__ __forceinline__ int parts_p(int rows, const Sizes& z) { return pieces(K == kForward8 ? rows : z.p, kTileP); }
template <Kind K>
__device__ __forceinline__ int parts_q(int rows, const Sizes& z)
{
  return K == kForward8 ? pieces(z.q, z.step) : pieces(K == kWeights ? z.q : rows, kTileQ);
}

template <Kind K>
__device__ __forceinline__ Tile tile_at(int t, const Sizes& z, const Control& sh)
{
  int low = 0, high = z.experts; // tile_start[low] <= t < tile_start[high]
  while (high - low > 1) {
    const int mid = (low + high) / 2;
    if (sh.tile_start[mid] <= t)
      low = mid;
    else
      high = mid;
  }
  Tile r;
  r.expert = low;
  r.row = sh.row_start[low];
  r.rows = sh.row_start[low + 1] - r.row;
  const int i = t - sh.tile_start[low];
  if constexpr (K == kForward8) {
    const int parts = parts_p<K>(r.rows, z);
    r.p = i % parts * kTileP;
    r.q = i / parts * z.step;
    r.width = min(z.step, z.q - r.q);
    r.blocks = pieces(z.c, 128);
  } else {
    const int q = K == kWeights ? z.q : r.rows;
    const int parts = parts_q<K>(r.rows, z);
    const int step = (pieces(q, parts) + 15) / 16 * 16;
    r.q = i % parts * step;
    r.width = min(step, q - r.q);
    r.p = i / parts * kTileP;
    r.blocks = K == kWeights ? pieces(r.rows, kDepth) : pieces(z.c, 64);
  }
  return r;
}

// join() of the values of the threads before this one (0 for the first), by
// all threads of the block.
template <class F>
__device__ int before_this_thread(int value, Control& sh, F&& join)
{
  const int lane = threadIdx.x & 31;
  int all = value;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int other = __shfl_up_sync(kAll, all, o);
    all = lane >= o ? join(all, other) : all;
  }
  if (lane == 31)
    sh.part[threadIdx.x / 32] = all;
  const int previous = __shfl_up_sync(kAll, all, 1);
  __syncthreads();
  int before = lane > 0 ? previous : 0;
  for (int w = 0; w < threadIdx.x / 32; ++w)
    before = join(before, sh.part[w]);
  __syncthreads();
  return before;
}

// The experts' first tiles and rows, by all threads of the block. Offsets out
// of range, or below an earlier one, are raised or lowered to the nearest that
// are not, so that no offsets lead outside the rows.
template <Kind K>
__device__ void find_tiles(const int64_t* offsets, const Sizes& z, Control& sh)
{
  constexpr int kMost = kMaxExperts / kThreads + 1; // offsets of a thread
  static_assert(kMost * kThreads > kMaxExperts);
  const int first = threadIdx.x * kMost;
  int row[kMost], most = 0;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int e = first + i;
    most = max(most, e <= z.experts ? (int)max(int64_t{0}, min(offsets[e], z.num_rows)) : 0);
    row[i] = most;
  }
  const int before = before_this_thread(most, sh, [](int a, int b) { return max(a, b); });
#pragma unroll
  for (int i = 0; i < kMost; ++i)
    if (first + i <= z.experts)
      sh.row_start[first + i] = max(row[i], before);
  __syncthreads();
  int tile[kMost], sum = 0;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int e = first + i;
    tile[i] = sum;
    if (e < z.experts) {
      const int rows = sh.row_start[e + 1] - sh.row_start[e];
      sum += parts_p<K>(rows, z) * parts_q<K>(rows, z);
    }
  }
  const int start = before_this_thread(sum, sh, [](int a, int b) { return a + b; });
#pragma unroll
  for (int i = 0; i < kMost; ++i)
    if (first + i <= z.experts)
      sh.tile_start[first + i] = start + tile[i];
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Kernel
// ---------------------------------------------------------------------------
constexpr bool eight(Kind k) { return k == kForward8; }
constexpr bool p_by_rows(Kind k) { return k == kForward8 || k == kForward; } // rows of c in shared memory
constexpr bool q_by_rows(Kind k) { return k != kWeights; }

// One thread: copies of the tiles' operands, as stages get free.
template <Kind K>
__device__ void copy_operands(const CUtensorMap& p_map, const CUtensorMap& q_map, const Sizes& z, char* stages, Control& sh)
{
  const int tiles = sh.tile_start[z.experts];
  Ring<kStages> s;
  int used = 0; // stages whose copies are under way or have landed
  bool ok = true;
  for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
    const Tile tile = tile_at<K>(t, z, sh);
    // boxes are copied whole, whatever of them there is
    const int boxes_p = K == kForward8 ? pieces(min(kTileP, tile.rows - tile.p), kBox) : 0;
    const int boxes_q = pieces(tile.width, K == kForward8 ? kTileP : q_by_rows(K) ? kBox : 64);
    const int bytes = K == kForward8 ? (boxes_p * kBox + boxes_q * kTileP) * 128
                                     : (kTileP + boxes_q * (q_by_rows(K) ? kBox : 64)) * 128;
    for (int b = 0; b < tile.blocks; ++b) {
      ok = wait(&sh.empty[s.at], s.parity ^ 1, sh);
      if (!ok)
        break;
      char *const to_p = stages + s.at * kStageBytes, *const to_q = to_p + kBytesP;
      uint64_t* const bar = &sh.full[s.at];
      mbar_arrive_expect_tx(bar, bytes);
      if constexpr (K == kForward8) {
        for (int i = 0; i < boxes_p; ++i)
          tile_load(to_p + i * kBox * 128, &p_map, b * 128, tile.row + tile.p + i * kBox, 0, bar);
        for (int i = 0; i < boxes_q; ++i)
          tile_load(to_q + i * kTileP * 128, &q_map, b * 128, tile.q + i * kTileP, tile.expert, bar);
      } else if constexpr (K == kWeights) {
        const int y = tile.row + b * kDepth;
        for (int i = 0; i < 2; ++i)
          tile_load(to_p + i * kDepth * 128, &p_map, tile.p + i * 64, y, 0, bar);
        for (int i = 0; i < boxes_q; ++i)
          tile_load(to_q + i * kDepth * 128, &q_map, tile.q + i * 64, y, 0, bar);
      } else {
        if constexpr (K == kForward)
          tile_load(to_p, &p_map, b * 64, tile.p, tile.expert, bar);
        else
          for (int i = 0; i < 2; ++i)
            tile_load(to_p + i * kDepth * 128, &p_map, tile.p + i * 64, b * kDepth, tile.expert, bar);
        for (int i = 0; i < boxes_q; ++i)
          tile_load(to_q + i * kBox * 128, &q_map, b * 64, tile.row + tile.q + i * kBox, 0, bar);
      }
      used = min(used + 1, kStages);
      s.next();
    }
  }
  if (!ok) {
    // what is under way lands before the block ends (a second each at most)
    for (int i = 0; i < used; ++i) {
      s.at = s.at == 0 ? kStages - 1 : s.at - 1;
      s.parity ^= s.at == kStages - 1;
      mbar_wait(&sh.full[s.at], s.parity);
    }
  }
}

// One warp: the products of the blocks that have landed.
template <Kind K>
__device__ void issue_products(const Sizes& z, char* stages, Control& sh)
{
  const int lane = threadIdx.x & 31, tiles = sh.tile_start[z.experts];
  const uint32_t tmem = sh.tmem;
  Ring<kStages> s;
  Ring<2> d;
  bool ok = true;
  for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
    const Tile tile = tile_at<K>(t, z, sh);
    const uint32_t instruction = z.instruction | (uint32_t)((tile.width + 15) / 16 * 2) << 17;
    for (int b = 0; b < tile.blocks; ++b) {
      // the sums of one block, or of all
      const bool first = eight(K) || b == 0, last = eight(K) || b == tile.blocks - 1;
      ok = (!first || wait(&sh.sums_empty[d.at], d.parity ^ 1, sh)) && wait(&sh.full[s.at], s.parity, sh);
      ok = __all_sync(kAll, ok);
      if (!ok)
        break;
      char* const from = stages + s.at * kStageBytes;
      if constexpr (K == kWeights) {
        // rows of the next expert, or of none, do not count
        const int left = tile.rows - b * kDepth;
        if (left < kDepth) {
          const int copies = 2 + pieces(tile.width, 64);
          for (int i = 0; i < copies; ++i)
            for (int at = left * 128 + lane * 16; at < kDepth * 128; at += 512)
              *reinterpret_cast<uint4*>(from + i * kDepth * 128 + at) = uint4{};
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
      }
      fence_after_sync();
      if (lane == 0) {
        const uint64_t p = operand<p_by_rows(K)>(smem_addr(from)), q = operand<q_by_rows(K)>(smem_addr(from) + kBytesP);
        // four products: 32 bytes of c on, or 16 rows of 128 bytes
#pragma unroll
        for (int i = 0; i < 4; ++i)
          multiply<eight(K)>(tmem + d.at * kTileQ, p + i * (p_by_rows(K) ? 2 : 128), q + i * (q_by_rows(K) ? 2 : 128),
                             instruction, !first || i > 0);
        commit(&sh.empty[s.at]);
        if (last)
          commit(&sh.sums_full[d.at]);
      }
      __syncwarp();
      s.next();
      if (last)
        d.next();
    }
  }
  if (!ok && lane == 0) {
    commit(&sh.drained); // what is under way ends before the block does
    mbar_wait(&sh.drained, 0);
  }
  __syncwarp();
}

// kSumWarps warps, 8-bit operands: each block's sums times their scales. A
// thread has one row, so one factor for all its columns of a block, which lie
// in one block of the weights' scales.
template <class O>
__device__ void add_scaled(const Sizes& z, O* out, Control& sh)
{
  const int warp = threadIdx.x / 32 - (kThreads / 32 - kSumWarps), lane = threadIdx.x & 31;
  const int quarter = warp & 3, start = warp / 4 * 128;
  const uint32_t lanes = sh.tmem + ((uint32_t)quarter * 32 << 16);
  const int tiles = sh.tile_start[z.experts];
  Ring<2> d;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Tile tile = tile_at<kForward8>(t, z, sh);
    const int mine = (tile.width - start + 31) / 32; // steps of 32 columns
    const int row = tile.p + quarter * 32 + lane;
    const bool on = row < tile.rows && mine > 0;
    const float* by_row = z.row_scales + (int64_t)(tile.row + row) * z.scale_stride;
    const float* by_weight =
      z.weight_scales + ((int64_t)tile.expert * pieces(z.q, 128) + (tile.q + start) / 128) * tile.blocks;
    float2 sum[64] = {};
    float scale = on ? by_row[0] * by_weight[0] : 0.0f;
    for (int b = 0; b < tile.blocks; ++b) {
      const float2 f = make_float2(scale, scale);
      if (on && b + 1 < tile.blocks)
        scale = by_row[b + 1] * by_weight[b + 1];
      if (!__all_sync(kAll, wait(&sh.sums_full[d.at], d.parity, sh)))
        return;
      fence_after_sync();
      const uint32_t from = lanes + d.at * kTileQ + start;
      uint32_t v[2][32];
      if (mine > 0)
        sums_load(v[0], from);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < mine) {
          sums_wait(v[c & 1]);
          if (c + 1 < mine)
            sums_load(v[(c + 1) & 1], from + (c + 1) * 32);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sum[c * 16 + i] =
              __ffma2_rn(make_float2(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1])), f,
                         sum[c * 16 + i]);
        }
      fence_before_sync();
      __syncwarp();
      if (lane == 0)
        arrive(&sh.sums_empty[d.at]);
      d.next();
    }
    if (on) {
      O* const to = out + (int64_t)(tile.row + row) * z.out_stride + tile.q + start;
      const int left = min(128, tile.width - start);
      if (z.out_vectors) { // left is a multiple of V
        constexpr int V = 16 / (int)sizeof(O);
#pragma unroll
        for (int c = 0; c < 128; c += V)
          if (c < left) {
            float x[V];
#pragma unroll
            for (int i = 0; i < V; i += 2)
              x[i] = sum[(c + i) / 2].x, x[i + 1] = sum[(c + i) / 2].y;
            store_f32<O, V>(to + c, x);
          }
      } else {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c < left)
            to[c] = from_f32<O>(c & 1 ? sum[c / 2].y : sum[c / 2].x);
      }
    }
  }
}

// kSumWarps warps, 16-bit operands: sums to memory. Lanes are neighbours
// there.
template <Kind K, class O>
__device__ void write_sums(const Sizes& z, O* out, Control& sh)
{
  const int warp = threadIdx.x / 32 - (kThreads / 32 - kSumWarps), lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const uint32_t lanes = sh.tmem + ((uint32_t)quarter * 32 << 16);
  const int tiles = sh.tile_start[z.experts];
  Ring<2> d;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Tile tile = tile_at<K>(t, z, sh);
    // half of the columns, in steps of 16
    const int steps = (tile.width + 15) / 16, steps0 = (steps + 1) / 2;
    const int start = warp < 4 ? 0 : steps0 * 16, mine = warp < 4 ? steps0 : steps - steps0;
    const int p = tile.p + quarter * 32 + lane;
    const int left = p < z.p ? tile.width - start : 0; // columns to write
    const int64_t row = K == kWeights ? (int64_t)tile.expert * z.q + tile.q : tile.row + tile.q;
    O* at = out + (row + start) * z.out_stride + p;
    const bool any = tile.blocks > 0; // none: an expert without rows has a gradient of zeros
    if (any) {
      if (!__all_sync(kAll, wait(&sh.sums_full[d.at], d.parity, sh)))
        return;
      fence_after_sync();
    }
    for (int c = 0; c < mine; ++c) {
      uint32_t v[16] = {};
      if (any) {
        sums_load(v, lanes + d.at * kTileQ + start + c * 16);
        sums_wait(v);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (c * 16 + i < left)
          *at = from_f32<O>(__uint_as_float(v[i]));
        at += z.out_stride;
      }
    }
    if (any) {
      fence_before_sync();
      __syncwarp();
      if (lane == 0)
        arrive(&sh.sums_empty[d.at]);
      d.next();
    }
  }
}

template <Kind K, class O>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
               const int64_t* offsets, const __grid_constant__ Sizes z, O* out)
{
  extern __shared__ char dynamic[];
  char* const stages = dynamic + (-smem_addr(dynamic) & 1023);
  Control& sh = *reinterpret_cast<Control*>(stages + kStages * kStageBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sums_full[i], 1);
      mbar_init(&sh.sums_empty[i], kSumWarps);
    }
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
    sh.failed = 0;
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    fence_before_sync();
  }
  wait_for_previous();
  allow_next();
  find_tiles<K>(offsets, z, sh); // ends with a barrier
  fence_after_sync();

  // With 8-bit operands a thread that adds up has 128 sums. What the other
  // warps give up of the 168 registers that each thread starts with, these
  // take: 128 * 72 + 256 * 216 = 384 * 168.
  if (warp < kThreads / 32 - kSumWarps) {
    if constexpr (eight(K))
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      if (lane == 0)
        copy_operands<K>(p_map, q_map, z, stages, sh);
    } else if (warp == 1) {
      issue_products<K>(z, stages, sh);
    }
  } else {
    if constexpr (eight(K)) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      add_scaled<O>(z, out, sh);
    } else {
      write_sums<K, O>(z, out, sh);
    }
    if constexpr (K != kWeights) {
      // rows that no expert has
      const int all = (int)gridDim.x * kSumWarps;
      const int first = (int)blockIdx.x * kSumWarps + warp - (kThreads / 32 - kSumWarps);
      for (int64_t r = sh.row_start[z.experts] + first; r < z.num_rows; r += all)
        for (int i = lane; i < z.out_stride; i += 32)
          out[r * z.out_stride + i] = from_f32<O>(0.0f);
    }
    fence_before_sync();
  }
  __syncthreads();
  if (warp == 2) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem));
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
using Encode = decltype(&cuTensorMapEncodeTiled);
Encode encoder()
{
  static const Encode found = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult what;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &what);
    return e == cudaSuccess && what == cudaDriverEntryPointSuccess ? (Encode)f : nullptr;
  }();
  return found;
}

// Matrices of `rows` rows of `width` elements of `size` bytes, `count` of
// them, in boxes of 128 bytes by `box` rows; zeros are read past the ends.
cudaError_t describe(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base, int64_t width, int64_t rows,
                     int64_t count, int64_t row_stride, int64_t stride, int box)
{
  const Encode encode = encoder();
  if (!encode)
    return cudaErrorSymbolNotFound;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)(row_stride * size), (cuuint64_t)(stride * size)};
  const cuuint32_t boxes[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box, 1}, steps[3] = {1, 1, 1};
  const CUresult r = encode(map, type, 3, const_cast<void*>(base), dims, strides, boxes, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The kernel's permission to use its shared memory belongs to each device's
// copy of it; asked for once a device.
template <Kind K, class O>
cudaError_t allow_shared()
{
  static std::atomic<uint64_t> done{0};
  int device;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess)
    return e;
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (done.load(std::memory_order_relaxed) & bit)
    return cudaSuccess;
  e = cudaFuncSetAttribute(product_kernel<K, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kShared);
  if (e == cudaSuccess)
    done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <Kind K, class O>
int run(const CUtensorMap& p, const CUtensorMap& q, const int64_t* offsets, const Sizes& z, void* out, int sms,
        int64_t most_tiles, void* stream)
{
  const cudaError_t e = allow_shared<K, O>();
  if (e != cudaSuccess)
    return record_cuda_error(e);
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(sms, most_tiles));
  return finish(launch(product_kernel<K, O>, dim3(grid), kThreads, kShared, (cudaStream_t)stream, p, q, offsets, z, (O*)out), 1);
}

bool float_type_of(int dtype) { return dtype == SEGTOPK_F16 || dtype == SEGTOPK_BF16 || dtype == SEGTOPK_F32; }

// Whether matrices can be described for TMA: 16-byte addresses and strides.
bool tma_fits(const void* p, int64_t stride, int size) { return aligned(p, 16) && stride * size % 16 == 0; }

constexpr int64_t kMaxSide = 1 << 20;
constexpr int64_t kMaxTiles = 1 << 30;
constexpr int64_t kMaxStride = 1ll << 36;

uint32_t instruction(int dtype, bool p_by_rows, bool q_by_rows) // sums in 32 bits, 128 lanes
{
  const uint32_t type = dtype == SEGTOPK_BF16 ? 1 : 0;
  return 1u << 4 | type << 7 | type << 10 | (uint32_t)!p_by_rows << 15 | (uint32_t)!q_by_rows << 16 |
         (uint32_t)(kTileP / 16) << 24;
}
CUtensorMapDataType map_type(int dtype)
{
  return dtype == SEGTOPK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

int check_sizes(int64_t num_rows, int64_t width, int64_t out_width, int32_t experts)
{
  if (num_rows < 0 || width < 1 || out_width < 1 || experts < 1)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (num_rows > 2147483647LL - kTileQ || width > kMaxSide || out_width > kMaxSide || experts > kMaxExperts)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  return SEGTOPK_SUCCESS;
}
// At most as many tiles there are of `by` rows and `by_out` outputs: an expert
// with r rows has at most r / by + 1 of each outputs, one without none.
int64_t forward_tiles(int64_t num_rows, int by, int64_t out_width, int by_out, int32_t experts)
{
  return (num_rows / by + std::min<int64_t>(experts, num_rows)) * ((out_width + by_out - 1) / by_out);
}

} // namespace

cudaError_t read_matmul_error(uint32_t* word)
{
  const uint32_t zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(word, g_device_error, sizeof(zero));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
}

} // namespace segtopk

using namespace segtopk;

extern "C" int segtopk_expert_matmul(segtopk_dtype dtype, const void* rows, int64_t num_rows, int64_t width,
                                     int64_t row_stride, const void* weights, int32_t experts, int64_t out_width,
                                     int64_t expert_stride, int64_t out_stride, int64_t in_stride,
                                     const int64_t* offsets, segtopk_dtype out_dtype, void* out, void* stream)
{
  record_launch_count(0);
  int rc = check_sizes(num_rows, width, out_width, experts);
  if (rc == SEGTOPK_ERROR_INVALID_VALUE || dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 || out_dtype < SEGTOPK_F16 ||
      out_dtype > SEGTOPK_I32 || (in_stride != 1 && out_stride != 1) || row_stride < width ||
      (in_stride == 1 && out_width > 1 ? out_stride < width : false) ||
      (in_stride != 1 && in_stride < out_width) || expert_stride < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  const bool turned = in_stride != 1;
  const int64_t line = turned ? in_stride : out_stride; // between rows of the weights in memory
  if (rc != SEGTOPK_SUCCESS || (dtype != SEGTOPK_F16 && dtype != SEGTOPK_BF16) || !float_type_of(out_dtype) ||
      width % 8 != 0 || (turned && out_width % 8 != 0) || row_stride > kMaxStride || line > kMaxStride ||
      expert_stride > kMaxStride || forward_tiles(num_rows, kTileQ, out_width, kTileP, experts) > kMaxTiles)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  if (num_rows == 0)
    return SEGTOPK_SUCCESS;
  if (!rows || !weights || !offsets || !out)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!tma_fits(rows, row_stride, 2) || !tma_fits(weights, line, 2) || expert_stride % 8 != 0 || !aligned(offsets, 8) ||
      !aligned(out, out_dtype == SEGTOPK_F32 ? 4 : 2))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  CUtensorMap p, q;
  cudaError_t e = turned ? describe(&p, map_type(dtype), 2, weights, out_width, width, experts, line, expert_stride, kDepth)
                         : describe(&p, map_type(dtype), 2, weights, width, out_width, experts, line, expert_stride, kTileP);
  if (e == cudaSuccess)
    e = describe(&q, map_type(dtype), 2, rows, width, num_rows, 1, row_stride, num_rows * row_stride, kBox);
  if (e != cudaSuccess)
    return record_cuda_error(e);
  Sizes z = {};
  z.num_rows = num_rows;
  z.experts = experts;
  z.p = (int)out_width;
  z.c = (int)width;
  z.instruction = instruction(dtype, !turned, true);
  z.out_stride = out_width;
  const int64_t tiles = forward_tiles(num_rows, kTileQ, out_width, kTileP, experts);
  return with_float_type(out_dtype, [&](auto zero) {
    using O = decltype(zero);
    return turned ? run<kForwardTurned, O>(p, q, offsets, z, out, sms, tiles, stream)
                  : run<kForward, O>(p, q, offsets, z, out, sms, tiles, stream);
  });
}

extern "C" int segtopk_expert_matmul_f8(const void* rows, int64_t num_rows, int64_t width, int64_t row_stride,
                                        const float* row_scales, int64_t scale_stride, const void* weights,
                                        int32_t experts, int64_t out_width, int64_t expert_stride, int64_t out_stride,
                                        const float* weight_scales, const int64_t* offsets, segtopk_dtype out_dtype,
                                        void* out, void* stream)
{
  record_launch_count(0);
  int rc = check_sizes(num_rows, width, out_width, experts);
  if (rc == SEGTOPK_ERROR_INVALID_VALUE || out_dtype < SEGTOPK_F16 || out_dtype > SEGTOPK_I32 || row_stride < width ||
      (out_width > 1 && out_stride < width) || expert_stride < 0 || scale_stride < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (rc != SEGTOPK_SUCCESS || !float_type_of(out_dtype) || width % 16 != 0 || row_stride > kMaxStride ||
      out_stride > kMaxStride || expert_stride > kMaxStride || forward_tiles(num_rows, kTileP, out_width, kTileP, experts) > kMaxTiles)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  if (num_rows == 0)
    return SEGTOPK_SUCCESS;
  if (!rows || !row_scales || !weights || !weight_scales || !offsets || !out)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!tma_fits(rows, row_stride, 1) || !tma_fits(weights, out_stride, 1) || expert_stride % 16 != 0 ||
      !aligned(offsets, 8) || !aligned(row_scales, 4) || !aligned(weight_scales, 4) ||
      !aligned(out, out_dtype == SEGTOPK_F32 ? 4 : 2))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  CUtensorMap p, q;
  cudaError_t e = describe(&p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, width, num_rows, 1, row_stride,
                           num_rows * row_stride, kBox);
  if (e == cudaSuccess)
    e = describe(&q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, weights, width, out_width, experts, out_stride, expert_stride,
                 kTileP);
  if (e != cudaSuccess)
    return record_cuda_error(e);
  // Tiles of 128 columns where those of 256 would leave SMs idle.
  const int step = forward_tiles(num_rows, kTileP, out_width, kTileQ, experts) < 2 * sms ? kTileP : kTileQ;
  const int64_t tiles = forward_tiles(num_rows, kTileP, out_width, step, experts);
  Sizes z = {};
  z.num_rows = num_rows;
  z.experts = experts;
  z.q = (int)out_width;
  z.c = (int)width;
  z.instruction = instruction(SEGTOPK_F16, true, true); // e4m3, as code 0 of 8-bit types
  z.out_stride = out_width;
  z.row_scales = row_scales;
  z.scale_stride = scale_stride;
  z.weight_scales = weight_scales;
  z.step = step;
  return with_float_type(out_dtype, [&](auto zero) {
    using O = decltype(zero);
    z.out_vectors = rows_fit(out, out_width, out_width, sizeof(O), 16 / (int)sizeof(O));
    return run<kForward8, O>(p, q, offsets, z, out, sms, tiles, stream);
  });
}

extern "C" int segtopk_expert_matmul_weights(segtopk_dtype dtype, const void* a_rows, int64_t a_width, int64_t a_stride,
                                             const void* b_rows, int64_t b_width, int64_t b_stride, int64_t num_rows,
                                             int32_t experts, const int64_t* offsets, segtopk_dtype out_dtype,
                                             void* out, void* stream)
{
  record_launch_count(0);
  int rc = check_sizes(num_rows, a_width, b_width, experts);
  if (rc == SEGTOPK_ERROR_INVALID_VALUE || dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 || out_dtype < SEGTOPK_F16 ||
      out_dtype > SEGTOPK_I32 || a_stride < a_width || b_stride < b_width)
    return SEGTOPK_ERROR_INVALID_VALUE;
  const int64_t tiles = (a_width + kTileQ - 1) / kTileQ * ((b_width + kTileP - 1) / kTileP) * experts;
  if (rc != SEGTOPK_SUCCESS || (dtype != SEGTOPK_F16 && dtype != SEGTOPK_BF16) || !float_type_of(out_dtype) ||
      a_width % 8 != 0 || b_width % 8 != 0 || a_stride > kMaxStride || b_stride > kMaxStride || tiles > kMaxTiles)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  if (!offsets || !out || (num_rows > 0 && (!a_rows || !b_rows)))
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!tma_fits(a_rows, a_stride, 2) || !tma_fits(b_rows, b_stride, 2) || !aligned(offsets, 8) ||
      !aligned(out, out_dtype == SEGTOPK_F32 ? 4 : 2))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  if (num_rows == 0) {
    const size_t bytes = (size_t)a_width * b_width * experts * (out_dtype == SEGTOPK_F32 ? 4 : 2);
    const cudaError_t e = cudaMemsetAsync(out, 0, bytes, (cudaStream_t)stream);
    return e == cudaSuccess ? SEGTOPK_SUCCESS : record_cuda_error(e);
  }
  CUtensorMap p, q;
  cudaError_t e = describe(&p, map_type(dtype), 2, b_rows, b_width, num_rows, 1, b_stride, num_rows * b_stride, kDepth);
  if (e == cudaSuccess)
    e = describe(&q, map_type(dtype), 2, a_rows, a_width, num_rows, 1, a_stride, num_rows * a_stride, kDepth);
  if (e != cudaSuccess)
    return record_cuda_error(e);
  Sizes z = {};
  z.num_rows = num_rows;
  z.experts = experts;
  z.p = (int)b_width;
  z.q = (int)a_width;
  z.instruction = instruction(dtype, false, false);
  z.out_stride = b_width;
  return with_float_type(out_dtype, [&](auto zero) {
    return run<kWeights, decltype(zero)>(p, q, offsets, z, out, sms, tiles, stream);
  });
}
