// Each expert's matrix product of its rows, and its gradients
// (segtopk_expert_matmul, segtopk_expert_matmul_f8 and
// segtopk_expert_matmul_weights in include/segtopk.h).
//
// All are products of tiles D[p, q] = sum_c P[p, c] Q[q, c] on the tensor cores
// (tcgen05), whose sums are held in 32 bits in tensor memory (TMEM): a lane for
// each p, a column for each q.
//   forward         p an expert's outputs, q its rows, c the width
//   rows' gradient  p an expert's inputs, q its rows, c the outputs: the
//                   forward product with the weights read the other way round
//   weights'        p and q an expert's inputs and outputs (the dense one of
//                   the weights as p), c its rows
//   8 bits          p an expert's rows, q its outputs, c the width
// In 16 bits the rows are q, since a tile may be any multiple of 32 of q wide:
// experts have as many rows as the router gives them, and a tile no more than
// that. In 8 bits the sum over one block of 128 values of c has one scale for
// each row and one for the weights' tile, so each block's sums are taken out
// of TMEM, multiplied and added up in registers in 32 bits; there the rows are
// p, which gives a lane one factor for all its columns (the other way round,
// with a factor a column from shared memory, a prefill took 3076 us instead of
// 1222).
//
// Two blocks on neighbouring SMs share a tile of 256 p by up to 256 q (pair()):
// each has half of p in its TMEM and copies half of q for both, which is what
// the way from L2 to an SM carries in the time of the products (64 bytes a
// cycle); one block alone on 128 p by 256 q needs half as much again. 8-bit
// rows of which an expert has few go to single blocks.
//
// Operands come by TMA in blocks of 128 bytes of c, six of them under way (192
// KB), four in a single block with its 256 q. Of a block's twelve warps one
// copies p, one q, one issues products and eight take sums out of TMEM, which
// holds two sets of them, so that one is taken out while the next is computed.
// Blocks stay on their SM and take tile after tile; each finds its tiles from
// the experts' offsets, which the host never reads.
//
// Measured on GB300 (two of them, through the Python API, results of the type of
// the rows, us): 20 calls one after the other, and the same calls for 4 s, which
// the GPU's power limit slows down.
//   16 bits, 8192^3, one expert                       592 to 611   692
//     cuBLAS                                          539 to 550   633
//   16 bits, 65536 rows of 128 experts, 2048x1024
//     forward                                         183 to 189   213
//     rows' gradient                                  187 to 192   217
//     weights' gradient                               226          251
//   8 bits, 131072 rows of 128 experts, 4096x2048     975 to 980   1056 to 1070
//   8 bits, 16384 rows of one expert, 8192x8192       864 to 888
//   8 bits, 64 rows of 64 experts, 2048x1024          17
// A block of the main loop takes 518 cycles of the tensor cores' 512 in the
// first. At the power limit its clock is 1.37 to 1.40 GHz, the library's 1.47 to
// 1.49: of the 9 % between the two 7 are the energy that a product takes here,
// and 2 cycles. In 8 bits a block takes 920 cycles: products that are issued back
// to back end that far apart while sums are loaded from TMEM, 530 while none are,
// and each block's 128 KB of sums have to be loaded. Whether TMEM carries no
// more, or the products wait for the release of one of the two sets, these
// figures do not tell apart. Beside that an expert's last tile of 256 rows is
// half empty on average, a ninth of the work at 1024 rows an expert. With few
// rows the weights' bytes bound it.
#include <atomic>
#include <cuda.h>

#include "common.cuh"
#include "expert_tiles.h"
#include "rows.cuh"

namespace segtopk {
namespace {
using namespace rows;

constexpr int kThreads = 384;
constexpr int kSumWarps = 8;     // of them the last
constexpr int kTileP = 128;      // of a block: the lanes of TMEM
constexpr int kOperandBytes = 192 << 10;
constexpr int kMaxStages = 6;
constexpr int kBytesP = kTileP * 128;
constexpr int kBox = 32;         // rows of one copy of few of an expert's rows
constexpr int kDepth = 64;       // rows of one copy where c runs over rows
constexpr int kProduct = 16;     // of them in one product
constexpr int kMaxExperts = SEGTOPK_MAX_EXPERTS;

enum Kind { kForward8, kForward8Pair, kForward, kForwardTurned, kWeights };
constexpr bool eight(Kind k) { return k == kForward8 || k == kForward8Pair; }
// Two blocks, of one cluster, on a tile: 256 p, half of them in each block's
// TMEM, and each reads half of the q for both.
constexpr bool pair(Kind k) { return k != kForward8; }
constexpr int blocks_of(Kind k) { return pair(k) ? 2 : 1; }
constexpr bool p_by_rows(Kind k) { return eight(k) || k == kForward; } // rows of c in shared memory
constexpr bool q_by_rows(Kind k) { return k != kWeights; }
constexpr int tile_p(Kind k) { return kTileP * blocks_of(k); }
constexpr int bytes_q(Kind k) { return kTileQ / blocks_of(k) * 128; }
constexpr int stage_bytes(Kind k) { return kBytesP + bytes_q(k); }
constexpr int stages_of(Kind k) { return kOperandBytes / stage_bytes(k); }
static_assert(stages_of(kForward) <= kMaxStages && stages_of(kForward8) <= kMaxStages);

struct Control {
  uint64_t full[kMaxStages], empty[kMaxStages]; // copies (a pair's: at its first block) have landed; products have read them
  uint64_t sums_full[2], sums_empty[2];         // TMEM's halves (empty: at the first block)
  uint64_t drained;                             // products behind a wait that ran out
  uint32_t tmem;
  int failed;                                   // a wait ran out: everybody leaves
  uint32_t progress;                            // kWeights: blocks of rows that this block has begun to copy
  long long wait_limit;                         // cycles
  int part[kThreads / 32];
  int tile_start[kMaxExperts + 1];              // experts' first tiles
  int row_start[kMaxExperts + 1];               // and rows
  uint4 staging[kSumWarps][32 * 4];             // 64 bytes of 32 rows on their way to memory
};
constexpr size_t kShared = 1024 + (size_t)kOperandBytes + sizeof(Control);
static_assert(kShared <= 227 * 1024, "shared memory of a block");

// Descriptors of the operands. kWeights: in boxes of kDepth rows, and for an
// expert's last rows of 8, 4, 2 and 1. Others: `large`, an expert's rows in
// boxes of kTileP, beside p or q in boxes of kBox.
constexpr int kEndBoxes = 4;
struct Maps {
  CUtensorMap p, q, large;
};
struct WeightsMaps {
  CUtensorMap p, q, p_end[kEndBoxes], q_end[kEndBoxes]; // of 8 >> i rows
};
template <Kind K>
using MapsOf = std::conditional_t<K == kWeights, WeightsMaps, Maps>;

struct Sizes {
  int64_t num_rows;     // slots; those before the first offset and from the last one on have no expert
  int experts;
  int p, q, c;          // sizes; an expert's rows take the place of one
  int step;             // 8 bits: the tiles' q
  uint32_t instruction; // types and majors of the operands
  int64_t out_stride;   // between rows of the result, which are dense
  bool out_vectors;     // its rows can be written 16 bytes at a time
  const float* row_scales;
  int64_t scale_stride;
  const float* weight_scales;
  long long wait_limit; // of a wait, in cycles
  int test_extra_bytes; // builds with test hooks: added to what a block's first copies are expected to bring
};

// ---------------------------------------------------------------------------
// Tensor memory and tensor cores
// ---------------------------------------------------------------------------
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// What follows is issued by one lane (`on`) of a warp whose lanes all get here:
// their operands then stay in the warp's uniform registers. In a branch that
// one lane takes alone each product cost 48 cycles and each copy 165.
__device__ __forceinline__ uint32_t elected()
{
  uint32_t on;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(on));
  return on;
}

// A copy that counts at `bar`: an address in the cluster's shared memory, of
// either block of a pair.
template <bool PAIR>
__device__ __forceinline__ void tile_load(uint32_t on, uint32_t to, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
#define SEGTOPK_COPY(GROUP)                                                                                      \
  asm volatile("{\n .reg .pred e;\n setp.ne.b32 e, %6, 0;\n"                                                    \
               " @e cp.async.bulk.tensor.3d" GROUP ".shared::cluster.global.tile.mbarrier::complete_tx::bytes "  \
               "[%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(to),                                                   \
               "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(on)                                               \
               : "memory")
  if constexpr (PAIR)
    SEGTOPK_COPY(".cta_group::2");
  else
    SEGTOPK_COPY("");
#undef SEGTOPK_COPY
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

template <Kind K>
__device__ __forceinline__ void multiply(uint32_t on, uint32_t sums, uint64_t p, uint64_t q, uint32_t instruction, bool add)
{
#define SEGTOPK_MULTIPLY(GROUP, TYPE)                                                                            \
  asm volatile("{\n .reg .pred a, e;\n setp.ne.b32 a, %4, 0;\n setp.ne.b32 e, %5, 0;\n"                         \
               " @e tcgen05.mma.cta_group::" GROUP ".kind::" TYPE " [%0], %1, %2, %3, a;\n}" ::"r"(sums),        \
               "l"(p), "l"(q), "r"(instruction), "r"((uint32_t)add), "r"(on)                                     \
               : "memory")
  if constexpr (eight(K) && pair(K))
    SEGTOPK_MULTIPLY("2", "f8f6f4");
  else if constexpr (eight(K))
    SEGTOPK_MULTIPLY("1", "f8f6f4");
  else
    SEGTOPK_MULTIPLY("2", "f16");
#undef SEGTOPK_MULTIPLY
}
// Arrives at `bar`, a pair's at both blocks', once the products issued so far
// are done.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t on, uint32_t bar)
{
  if constexpr (PAIR)
    asm volatile("{\n .reg .pred e;\n setp.ne.b32 e, %2, 0;\n @e tcgen05.commit.cta_group::2.mbarrier::arrive::one"
                 ".shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(bar),
                 "h"((uint16_t)3), "r"(on)
                 : "memory");
  else
    asm volatile("{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n @e tcgen05.commit.cta_group::1.mbarrier::arrive::one"
                 ".shared::cluster.b64 [%0];\n}" ::"r"(bar),
                 "r"(on)
                 : "memory");
}
__device__ __forceinline__ void expect(uint32_t on, uint32_t bar, int bytes)
{
  asm volatile("{\n .reg .pred e;\n setp.ne.b32 e, %2, 0;\n @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(bar),
               "r"(bytes), "r"(on)
               : "memory");
}
// At a barrier of either block of a pair: that this warp's loads from TMEM are
// done, so that products of the first block may write there. The fences for
// TMEM around it (fence_before_sync, fence_after_sync) and the scope of the
// cluster order the two; no memory is handed over, so it is no release, which
// waits until all of the block's writes are visible everywhere: once every block
// of 8-bit operands that doubled the time of a product.
__device__ __forceinline__ void arrive(uint32_t bar)
{
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The address of the first block's `bar`.
template <Kind K>
__device__ __forceinline__ uint32_t at_first(uint64_t* bar)
{
  return pair(K) ? dsmem_map(smem_addr(bar), 0) : smem_addr(bar);
}
template <Kind K>
__device__ __forceinline__ int rank() // in the pair
{
  return pair(K) ? (int)(blockIdx.x & 1) : 0;
}

// Columns of this warp's 32 lanes. Load and wait are one statement: values
// that pass through a second one as operands were copied, 64 of them, which
// took longer than the products.
__device__ __forceinline__ void sums_load(uint32_t (&v)[64], uint32_t at)
{
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
               "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, "
               "%38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, "
               "%56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                 "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                 "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
                 "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
                 "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]),
                 "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), "=r"(v[40]), "=r"(v[41]), "=r"(v[42]),
                 "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]), "=r"(v[48]), "=r"(v[49]),
                 "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]), "=r"(v[56]),
                 "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
               : "r"(at)
               : "memory");
}

// TMEM: for an arrive(), which hands over TMEM alone.
template <bool TMEM>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity)
{
  uint32_t ok;
#define SEGTOPK_WAIT(HOW)                                                                                        \
  asm volatile("{\n .reg .pred p;\n mbarrier." HOW ".shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"   \
               : "=r"(ok)                                                                                        \
               : "r"(bar), "r"(parity)                                                                           \
               : "memory")
  if constexpr (TMEM)
    SEGTOPK_WAIT("try_wait.parity.relaxed.cluster");
  else
    SEGTOPK_WAIT("try_wait.parity");
  return ok != 0;
}
// One warp: waits for the phase of `bar` with this parity; false, for good,
// after about a second, or once another wait of the block has run out. A
// LONG wait lasts as long as an expert has rows: its second begins anew as
// long as the block goes on to copy.
template <bool LONG = false, bool TMEM = false>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Control& sh)
{
  if (__all_sync(kAll, try_wait<TMEM>(bar, parity)))
    return true;
  long long start = clock64();
  uint32_t seen = LONG ? *(volatile uint32_t*)&sh.progress : 0;
  bool failed = false;
  while (!__all_sync(kAll, try_wait<TMEM>(bar, parity))) {
    if (clock64() - start > sh.wait_limit) {
      const uint32_t now = LONG ? *(volatile uint32_t*)&sh.progress : 0;
      if (now != seen) {
        seen = now;
        start = clock64();
      } else {
        *(volatile int*)&sh.failed = 1;
        raise_error(kErrCopyTimeout);
      }
    }
    failed = *(volatile int*)&sh.failed;
    if (__any_sync(kAll, failed))
      return false;
  }
  return true;
}
template <bool LONG = false>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Control& sh)
{
  return wait<LONG>(smem_addr(bar), parity, sh);
}

// Whether that phase is over already; does not wait. Asked a step ahead, so
// that the answer is there when the step comes.
template <bool TMEM = false>
__device__ __forceinline__ bool over(uint32_t bar, uint32_t parity)
{
  uint32_t ok;
  if constexpr (TMEM)
    SEGTOPK_WAIT("test_wait.parity.relaxed.cluster");
  else
    SEGTOPK_WAIT("test_wait.parity");
  return ok != 0;
}
#undef SEGTOPK_WAIT

// The same value in all lanes, known to be so.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(kAll, x); }

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
struct Tile {
  int expert;
  int p;          // first
  int q, width;   // first and how many; kStepQ times as many as hold them are computed
  int row, rows;  // the expert's rows
  int blocks;     // of c
};

// Tiles of an expert with this many rows. Where q are its rows, or its inputs
// or outputs, it goes to as few tiles as hold it (even_part()).
template <Kind K>
__device__ __forceinline__ int parts_p(int rows, const Sizes& z) { return pieces(eight(K) ? rows : z.p, tile_p(K)); }
template <Kind K>
__device__ __forceinline__ int parts_q(int rows, const Sizes& z)
{
  return eight(K) ? pieces(z.q, z.step) : pieces(K == kWeights ? z.q : rows, kTileQ);
}

// Tile t, by a whole warp, which finds its expert in two looks: among every
// 32nd, then the 32 after that.
template <Kind K>
__device__ __forceinline__ Tile tile_at(int t, const Sizes& z, const Control& sh)
{
  static_assert(kMaxExperts <= 32 * 32);
  const int lane = threadIdx.x & 31;
  const int far = (lane + 1) * 32;
  const int base = 32 * __popc(__ballot_sync(kAll, far < z.experts && sh.tile_start[min(far, kMaxExperts)] <= t));
  const int near = base + lane;
  const int low = base + __popc(__ballot_sync(kAll, near < z.experts && sh.tile_start[min(near + 1, kMaxExperts)] <= t));
  Tile r;
  r.expert = low;
  r.row = sh.row_start[low];
  r.rows = sh.row_start[low + 1] - r.row;
  const int i = t - sh.tile_start[low];
  if constexpr (eight(K)) {
    const int parts = parts_p<K>(r.rows, z), q = divide(i, parts);
    r.p = (i - q * parts) * tile_p(K);
    r.q = q * z.step;
    r.width = min(z.step, z.q - r.q);
    r.blocks = pieces(z.c, 128);
  } else {
    const int q = K == kWeights ? z.q : r.rows;
    const int parts = parts_q<K>(r.rows, z);
    const int p = divide(i, parts);
    const TilePart part = even_part(q, parts, i - p * parts);
    r.q = part.first;
    r.width = part.width;
    r.p = p * tile_p(K);
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
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) { // all are read at once
    const int part = sh.part[w];
    before = w < threadIdx.x / 32 ? join(before, part) : before;
  }
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
// A warp each for p and q: copies of this block's operands, as stages get
// free. A pair's count at the first block, whose warp for p expects those of
// both; they may land before it says so, since the phase waits for that too.
// An expert's rows come in boxes of kTileP, or of kBox where that is less; all
// boxes are copied whole, whatever of them there is.
//
// kWeights: an expert's last block of rows has `left` of them, and the products
// read that many in steps of kProduct. Those rows are copied in boxes of 8, 4, 2
// and 1, and the ones up to the step from behind the tensor, where zeros are
// read; so the rows of the next expert, or of none, never get here.
// 65536 rows of 128 experts, 2048x1024: 226 us. (Copied whole, with zeros
// written over them by each block for the products of both, they need a release
// at cluster scope between the two, which also waits for results on their way
// to memory: 253 us, and 220 without it, which nothing in the order of memory
// allows.)
__device__ __forceinline__ int boxed(int rows) { return rows > kTileP / 2 ? kTileP : pieces(max(rows, 0), kBox) * kBox; }

template <Kind K, bool IS_P>
__device__ void copy_operands(const MapsOf<K>& maps, const Sizes& z, char* stages, Control& sh)
{
  constexpr int kStages = stages_of(K);
  constexpr bool kByRows = IS_P == eight(K) && K != kWeights; // these are the expert's rows
  const int tiles = uniform(sh.tile_start[z.experts]), me = rank<K>();
  const uint32_t on = elected(), to = smem_addr(stages) + (IS_P ? 0 : kBytesP);
  const uint32_t full = at_first<K>(&sh.full[0]), empty = smem_addr(&sh.empty[0]);
  Ring<kStages> s;
  const CUtensorMap& map = IS_P ? maps.p : maps.q;
  int used = 0;       // stages whose copies are under way or have landed
  uint32_t begun = 0; // kWeights: blocks of rows
  bool ok = true, ready = false;
  for (int t = blockIdx.x / blocks_of(K); ok && t < tiles; t += gridDim.x / blocks_of(K)) {
    const Tile tile = tile_at<K>(t, z, sh);
    const int width = pieces(tile.width, kStepQ) * kStepQ / blocks_of(K); // of q in this block
    // rows of 128 bytes that land
    int lines_p = kTileP, lines_q;
    if constexpr (eight(K)) {
      lines_p = boxed(tile.rows - tile.p - me * kTileP);
      lines_q = pieces(width, kTileP) * kTileP;
    } else {
      lines_q = K == kWeights ? pieces(width, 64) * 64 : boxed(width);
    }
    const int landing = uniform((lines_p + lines_q) * 128);
    int expected = landing;
    if constexpr (pair(K))
      expected += eight(K) ? (boxed(tile.rows - tile.p - kTileP) + lines_q) * 128 : landing;
    expected = uniform(expected);
    const int lines = uniform(IS_P ? lines_p : lines_q);
    const bool whole = kByRows && lines == kTileP;
    const int box = K == kWeights || (IS_P && K == kForwardTurned) ? 64 : kByRows && !whole ? kBox : kTileP;
    const int first = uniform((IS_P ? tile.p + me * kTileP : tile.q + me * width) + (kByRows ? tile.row : 0));
    const int row = uniform(tile.row), matrix = uniform(kByRows ? 0 : tile.expert), blocks = uniform(tile.blocks);
    const int left = uniform(K == kWeights ? tile.rows % kDepth : 0); // rows of the last block, if not all
    for (int b = 0; b < blocks; ++b) {
      if (!__all_sync(kAll, ready))
        ok = wait(empty + s.at * 8, s.parity ^ 1, sh);
      if (!ok)
        break;
      if (K == kWeights && IS_P)
        *(volatile uint32_t*)&sh.progress = ++begun; // by all lanes, the same
#ifdef SEGTOPK_TEST_HOOKS
      const int extra = used == 0 ? z.test_extra_bytes : 0;
#else
      constexpr int extra = 0;
#endif
      const uint32_t bar = full + s.at * 8, at = to + s.at * stage_bytes(K);
      const bool end = K == kWeights && left > 0 && b == blocks - 1;
      if (IS_P && me == 0)
        expect(on, bar, (end ? expected / (kDepth / kProduct) * pieces(left, kProduct) : expected) + extra);
      used = min(used + 1, kStages);
      s.next();
      ready = over(empty + s.at * 8, s.parity ^ 1);
      if constexpr (K == kWeights) {
        if (!end) {
          for (int i = 0; i < lines; i += 64)
            tile_load<true>(on, at + i * 128, &map, first + i, row + b * kDepth, 0, bar);
        } else {
          const CUtensorMap* const boxes = IS_P ? maps.p_end : maps.q_end;
          for (int i = 0; i < lines; i += 64) {
            int r = 0;
            auto copy = [&](int box, int y) {
              tile_load<true>(on, at + (i + r) * 128, &boxes[box], first + i, y, 0, bar);
              r += 8 >> box;
            };
            while (r + 8 <= left)
              copy(0, row + b * kDepth + r);
#pragma unroll
            for (int box = 1; box < kEndBoxes; ++box)
              if (left & 8 >> box)
                copy(box, row + b * kDepth + r);
#pragma unroll
            for (int box = kEndBoxes - 1; box >= 0; --box) // 8 is half of kProduct
              if (r & 8 >> box)
                copy(box, (int)z.num_rows);
          }
        }
      } else if constexpr (K == kForwardTurned && IS_P) {
#pragma unroll
        for (int i = 0; i < kTileP; i += 64)
          tile_load<true>(on, at + i * 128, &map, first + i, b * kDepth, matrix, bar);
      } else if (whole) {
        tile_load<pair(K)>(on, at, &maps.large, b * (eight(K) ? 128 : 64), first, 0, bar);
      } else {
        for (int i = 0; i < lines; i += box)
          tile_load<pair(K)>(on, at + i * 128, &map, b * (eight(K) ? 128 : 64), first + i, matrix, bar);
      }
    }
  }
  if (!ok && IS_P && me == 0) {
    // what is under way lands before the blocks end (a second each at most)
    for (int i = 0; i < used; ++i) {
      s.at = s.at == 0 ? kStages - 1 : s.at - 1;
      s.parity ^= s.at == kStages - 1;
      mbar_wait(&sh.full[s.at], s.parity, sh.wait_limit);
    }
  }
}

// One warp, of a pair's first block: the products of the blocks that have
// landed.
template <Kind K>
__device__ void issue_products(const Sizes& z, char* stages, Control& sh)
{
  const int tiles = uniform(sh.tile_start[z.experts]);
  const uint32_t on = elected(), tmem = uniform(sh.tmem);
  const uint64_t p0 = operand<p_by_rows(K)>(smem_addr(stages)), q0 = operand<q_by_rows(K)>(smem_addr(stages) + kBytesP);
  const uint32_t full = smem_addr(&sh.full[0]), empty = smem_addr(&sh.empty[0]), sums_full = smem_addr(&sh.sums_full[0]),
                 sums_empty = smem_addr(&sh.sums_empty[0]);
  Ring<stages_of(K)> s;
  Ring<2> d;
  bool ok = true, ready = false, sums_ready = false;
  for (int t = blockIdx.x / blocks_of(K); ok && t < tiles; t += gridDim.x / blocks_of(K)) {
    const Tile tile = tile_at<K>(t, z, sh);
    const uint32_t instruction = uniform((int)(z.instruction | (uint32_t)(pieces(tile.width, kStepQ) * kStepQ / 8) << 17));
    const int blocks = uniform(tile.blocks);
    // four products: 32 bytes of c on, or 16 rows of 128 bytes; an expert's last rows may be fewer
    const int last_products = uniform(K == kWeights && tile.rows > 0 ? pieces(tile.rows - (blocks - 1) * kDepth, kProduct) : 4);
    for (int b = 0; b < blocks; ++b) {
      // the sums of one block, or of all
      const bool first = eight(K) || b == 0, last = eight(K) || b == blocks - 1;
      if (first && !__all_sync(kAll, sums_ready))
        ok = wait<false, true>(sums_empty + d.at * 8, d.parity ^ 1, sh);
      if (ok && !__all_sync(kAll, ready))
        ok = wait(full + s.at * 8, s.parity, sh);
      if (!ok)
        break;
      fence_after_sync();
      const uint64_t p = p0 + s.at * (stage_bytes(K) / 16), q = q0 + s.at * (stage_bytes(K) / 16);
      const uint32_t sums = tmem + d.at * kTileQ, free = empty + s.at * 8, done = sums_full + d.at * 8;
      s.next();
      ready = over(full + s.at * 8, s.parity);
      if (last) {
        d.next();
        sums_ready = over<true>(sums_empty + d.at * 8, d.parity ^ 1);
      }
      const int products = K == kWeights && b == blocks - 1 ? last_products : 4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (K != kWeights || i < products)
          multiply<K>(on, sums, p + i * (p_by_rows(K) ? 2 : 128), q + i * (q_by_rows(K) ? 2 : 128), instruction,
                      !first || i > 0);
      commit<pair(K)>(on, free);
      if (last)
        commit<pair(K)>(on, done);
    }
  }
  if (!ok) {
    commit<pair(K)>(on, smem_addr(&sh.drained)); // what is under way ends before the blocks do
    if (on)
      mbar_wait(&sh.drained, 0, sh.wait_limit);
  }
  __syncwarp();
}

// A warp's 32 rows, one a lane, of `columns` values to memory, `stride` apart
// from `to` on; the first `rows` of them. They pass through shared memory 64
// bytes at a time, so that lanes write a row together: four of them 16 bytes
// each with rows on 16-byte boundaries, else one for each value. A store whose
// lanes write to a row each takes 32 cycles of an SM's memory pipe; with 16
// bytes a lane a tile's took longer than four of its blocks' products, with a
// value a lane the whole product four times as long.
template <class O, int N, class F>
__device__ __forceinline__ void write_rows(O* to, int64_t stride, int rows, int columns, bool vectors, uint4* staging, F&& sum)
{
  constexpr int V = 16 / (int)sizeof(O);
  const int lane = threadIdx.x & 31;
  auto place = [](int row, int u) { return row * 4 + (u ^ (row >> 1 & 3)); }; // eight lanes in different banks
  if (vectors) { // columns is a multiple of V
    const int unit = lane & 3;
#pragma unroll
    for (int c = 0; c < N; c += 4 * V) {
      if (c >= columns)
        break;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
          x[i] = sum(c + u * V + i);
        Vec<O, V> v;
        v.set(x);
        staging[place(lane, u)] = *reinterpret_cast<const uint4*>(&v);
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = j * 8 + lane / 4;
        const uint4 v = staging[place(row, unit)];
        if (row < rows && c + unit * V < columns)
          *reinterpret_cast<uint4*>(to + row * stride + c + unit * V) = v;
      }
      __syncwarp();
    }
  } else {
    O* const values = reinterpret_cast<O*>(staging);
    const int i = lane % (4 * V);
#pragma unroll
    for (int c = 0; c < N; c += 4 * V) {
      if (c >= columns)
        break;
#pragma unroll
      for (int k = 0; k < 4 * V; ++k)
        values[lane * 4 * V + (k ^ (lane & (4 * V - 1)))] = from_f32<O>(sum(c + k));
      __syncwarp();
      for (int row = lane / (4 * V); row < min(rows, 32); row += 32 / (4 * V))
        if (c + i < columns)
          to[row * stride + c + i] = values[row * 4 * V + (i ^ (row & (4 * V - 1)))];
      __syncwarp();
    }
  }
}

// kSumWarps warps, 8-bit operands: each block's sums times their scales. A
// thread has one row, so one factor for all its columns of a block, which lie
// in one block of the weights' scales.
template <Kind K, class O>
__device__ void add_scaled(const Sizes& z, O* out, Control& sh)
{
  const int warp = threadIdx.x / 32 - (kThreads / 32 - kSumWarps), lane = threadIdx.x & 31;
  const int quarter = warp & 3, start = warp / 4 * 128;
  const uint32_t lanes = sh.tmem + ((uint32_t)quarter * 32 << 16);
  const int tiles = sh.tile_start[z.experts];
  Ring<2> d;
  for (int t = blockIdx.x / blocks_of(K); t < tiles; t += gridDim.x / blocks_of(K)) {
    const Tile tile = tile_at<K>(t, z, sh);
    const int columns = tile.width - start; // the rest of them
    const int row = tile.p + rank<K>() * kTileP + quarter * 32 + lane;
    const bool on = row < tile.rows && columns > 0;
    const float* by_row = z.row_scales + (int64_t)(tile.row + row) * z.scale_stride;
    const float* by_weight =
      z.weight_scales + ((int64_t)tile.expert * pieces(z.q, 128) + (tile.q + start) / 128) * tile.blocks;
    float2 sum[64] = {};
    float scale = on ? by_row[0] * by_weight[0] : 0.0f;
    for (int b = 0; b < tile.blocks; ++b) {
      const float2 f = make_float2(scale, scale);
      if (on && b + 1 < tile.blocks)
        scale = by_row[b + 1] * by_weight[b + 1];
      if (!wait(&sh.sums_full[d.at], d.parity, sh))
        return;
      fence_after_sync();
      const uint32_t from = lanes + d.at * kTileQ + start;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (columns <= 0)
          break;
        uint32_t v[64];
        sums_load(v, from + c * 64);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          sum[c * 32 + i] =
            __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f, sum[c * 32 + i]);
      }
      // (said right after the second load, before its products, this took 9 %
      // more: registers were spilled)
      fence_before_sync();
      __syncwarp();
      if (lane == 0)
        arrive(at_first<K>(&sh.sums_empty[d.at]));
      d.next();
    }
    const int first = row - lane; // of the warp
    if (columns > 0 && first < tile.rows)
      write_rows<O, 128>(out + (int64_t)(tile.row + first) * z.out_stride + tile.q + start, z.out_stride, tile.rows - first,
                         min(128, columns), z.out_vectors, sh.staging[warp],
                         [&](int i) { return i & 1 ? sum[i / 2].y : sum[i / 2].x; });
  }
}

// A warp's 32 columns of a 16-bit result, of which a lane has 32 rows' values,
// to memory, `stride` between rows: the first `rows` rows, `lanes` columns.
// Pairs of rows pass through shared memory, so that four lanes write 64 bytes
// of a row. Written by a store a row, two bytes a lane, a tile of 256 by 256
// took 5400 cycles, as long as ten blocks' products.
template <class O, class F>
__device__ __forceinline__ void write_columns(O* to, int64_t stride, int rows, int lanes, uint4* staging, F&& sum)
{
  const int lane = threadIdx.x & 31, unit = lane & 3;
  uint32_t* const words = reinterpret_cast<uint32_t*>(staging); // [pair of rows][column]: the values of both
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    Vec<O, 2> v;
    v.set({sum(2 * k), sum(2 * k + 1)});
    words[k * 32 + lane] = v.w[0];
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int k = j * 8 + lane / 4;
    // eight columns' pairs, in an order that takes eight lanes to different banks
    const uint4* const from = staging + k * 8 + unit * 2;
    const uint4 x = from[k & 1], y = from[~k & 1];
    const uint4 a = k & 1 ? y : x, b = k & 1 ? x : y;
    if (unit * 8 < lanes) {
      O* const at = to + 2 * k * stride + unit * 8;
      if (2 * k < rows)
        *reinterpret_cast<uint4*>(at) = {__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                         __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410)};
      if (2 * k + 1 < rows)
        *reinterpret_cast<uint4*>(at + stride) = {__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                                  __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632)};
    }
  }
  __syncwarp();
}

// kSumWarps warps, 16-bit operands: sums to memory, where the neighbours of a
// lane's value are the other lanes'. The weights' gradient with the operands
// exchanged, so that a lane stores 16 bytes of a row of its own, took 302 us
// where a store of two bytes a lane took 237 (65536 rows of 128 experts,
// 2048x1024).
template <Kind K, class O>
__device__ void write_sums(const Sizes& z, O* out, Control& sh)
{
  const int warp = threadIdx.x / 32 - (kThreads / 32 - kSumWarps), lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const uint32_t lanes = sh.tmem + ((uint32_t)quarter * 32 << 16);
  const int tiles = sh.tile_start[z.experts];
  Ring<2> d;
  for (int t = blockIdx.x / blocks_of(K); t < tiles; t += gridDim.x / blocks_of(K)) {
    const Tile tile = tile_at<K>(t, z, sh);
    // half of the columns, in steps of 16
    const int steps = (tile.width + 15) / 16, steps0 = (steps + 1) / 2;
    const int start = warp < 4 ? 0 : steps0 * 16;
    const int columns = warp < 4 ? min(steps0 * 16, tile.width) : tile.width - start;
    const int p = tile.p + rank<K>() * kTileP + quarter * 32 + lane;
    const bool any = tile.blocks > 0; // none: an expert without rows has a gradient of zeros
    if (any) {
      if (!wait<K == kWeights>(&sh.sums_full[d.at], d.parity, sh))
        return;
      fence_after_sync();
    }
    const uint32_t from = lanes + d.at * kTileQ + start;
    const int64_t row = K == kWeights ? (int64_t)tile.expert * z.q + tile.q : tile.row + tile.q;
    O* at = out + (row + start) * z.out_stride + p;
    const int left = p < z.p ? columns : 0;
    for (int c = 0; c < columns; c += 64) {
      uint32_t v[64] = {};
      if (any)
        sums_load(v, from + c);
      if (sizeof(O) == 2 && z.out_vectors) {
        if constexpr (sizeof(O) == 2)
#pragma unroll
          for (int i = 0; i < 64; i += 32)
            write_columns(at - lane + (c + i) * z.out_stride, z.out_stride, columns - c - i, z.p - (p - lane), sh.staging[warp],
                          [&](int k) { return __uint_as_float(v[i + k]); });
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (c + i < left)
            at[(c + i) * z.out_stride] = from_f32<O>(__uint_as_float(v[i]));
      }
    }
    if (any) {
      fence_before_sync();
      __syncwarp();
      if (lane == 0)
        arrive(at_first<K>(&sh.sums_empty[d.at]));
      d.next();
    }
  }
}

template <Kind K, class O>
__global__ void __cluster_dims__(blocks_of(K), 1, 1) __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ MapsOf<K> maps, const int64_t* offsets, const __grid_constant__ Sizes z, O* out)
{
  extern __shared__ char dynamic[];
  char* const stages = dynamic + (-smem_addr(dynamic) & 1023);
  Control& sh = *reinterpret_cast<Control*>(stages + kOperandBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

  if (threadIdx.x == 32)
    for (size_t i = 0; i < sizeof(maps) / sizeof(CUtensorMap); ++i)
      asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.p + i));
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sums_full[i], 1);
      mbar_init(&sh.sums_empty[i], kSumWarps * blocks_of(K));
    }
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
    sh.failed = 0;
    sh.progress = 0;
    sh.wait_limit = z.wait_limit;
  }
  if (warp == 2) {
    if constexpr (pair(K)) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before_sync();
  }
  wait_for_previous();
  allow_next();
  find_tiles<K>(offsets, z, sh); // ends with a barrier
  if constexpr (pair(K))
    cluster_sync(); // the other block's barriers are there too
  fence_after_sync();

  // With 8-bit operands a thread that adds up has 128 sums. What the other
  // warps give up of the 168 registers that each thread starts with, these
  // take: 128 * 72 + 256 * 216 = 384 * 168.
  if (warp < kThreads / 32 - kSumWarps) {
    if constexpr (eight(K))
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      copy_operands<K, true>(maps, z, stages, sh);
    } else if (warp == 3) {
      copy_operands<K, false>(maps, z, stages, sh);
    } else if (warp == 1) {
      if (rank<K>() == 0)
        issue_products<K>(z, stages, sh);
    }
  } else {
    if constexpr (eight(K)) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      add_scaled<K, O>(z, out, sh);
    } else {
      write_sums<K, O>(z, out, sh);
    }
    if constexpr (K != kWeights) {
      // rows that no expert has
      const int all = (int)gridDim.x * kSumWarps;
      const int begin = sh.row_start[0], end = sh.row_start[z.experts];
      const int64_t rows = begin + (z.num_rows - end);
      for (int64_t i = (int)blockIdx.x * kSumWarps + warp - (kThreads / 32 - kSumWarps); i < rows; i += all) {
        O* const to = out + free_row(begin, end, i) * z.out_stride;
        for (int c = lane; c < z.out_stride; c += 32)
          to[c] = from_f32<O>(0.0f);
      }
    }
    fence_before_sync();
  }
  __syncwarp();
  if constexpr (pair(K))
    cluster_sync(); // nothing arrives here or reads from here any more
  else
    __syncthreads();
  if (warp == 2) {
    fence_after_sync();
    if constexpr (pair(K))
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem));
    else
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
// them, in boxes of 128 bytes by `box` rows; zeros are read past the ends. The
// distance of a single one says nothing, but is described too.
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
int run(const MapsOf<K>& maps, const int64_t* offsets, Sizes z, void* out, int sms, int64_t most_tiles, void* stream)
{
  uint32_t extra;
  test_hooks(&z.wait_limit, &extra);
  z.test_extra_bytes = (int)extra;
  const cudaError_t e = allow_shared<K, O>();
  if (e != cudaSuccess)
    return record_cuda_error(e);
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(sms / blocks_of(K), most_tiles)) * blocks_of(K);
  return finish(launch(product_kernel<K, O>, dim3(grid), kThreads, kShared, (cudaStream_t)stream, maps, offsets, z, (O*)out), 1);
}

bool float_type_of(int dtype) { return dtype == SEGTOPK_F16 || dtype == SEGTOPK_BF16 || dtype == SEGTOPK_F32; }

// Whether matrices can be described for TMA: 16-byte addresses and strides.
bool tma_fits(const void* p, int64_t stride, int size) { return aligned(p, 16) && stride * size % 16 == 0; }

constexpr int64_t kMaxSide = 1 << 20;
constexpr int64_t kMaxTiles = 1 << 30;
constexpr int64_t kMaxStride = 1ll << 36;

// Sums in 32 bits; type: 0 for f16 and e4m3, 1 for bf16.
uint32_t instruction(Kind k, uint32_t type)
{
  return 1u << 4 | type << 7 | type << 10 | (uint32_t)!p_by_rows(k) << 15 | (uint32_t)!q_by_rows(k) << 16 |
         (uint32_t)(tile_p(k) / 16) << 24;
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
      (in_stride == 1 ? out_width > 1 && out_stride < width : in_stride < out_width) ||
      (rc == SEGTOPK_SUCCESS && experts > 1 && expert_stride < width * out_width))
    return SEGTOPK_ERROR_INVALID_VALUE;
  const bool turned = in_stride != 1;
  // between rows of the weights in memory, and matrices; those of one say nothing
  const int64_t line = turned ? in_stride : out_width > 1 ? out_stride : width;
  if (experts == 1)
    expert_stride = line;
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
  Maps maps;
  cudaError_t e = turned ? describe(&maps.p, map_type(dtype), 2, weights, out_width, width, experts, line, expert_stride, kDepth)
                         : describe(&maps.p, map_type(dtype), 2, weights, width, out_width, experts, line, expert_stride, kTileP);
  if (e == cudaSuccess)
    e = describe(&maps.q, map_type(dtype), 2, rows, width, num_rows, 1, row_stride, row_stride, kBox);
  if (e == cudaSuccess)
    e = describe(&maps.large, map_type(dtype), 2, rows, width, num_rows, 1, row_stride, row_stride, kTileP);
  if (e != cudaSuccess)
    return record_cuda_error(e);
  Sizes z = {};
  z.num_rows = num_rows;
  z.experts = experts;
  z.p = (int)out_width;
  z.c = (int)width;
  z.instruction = instruction(turned ? kForwardTurned : kForward, dtype == SEGTOPK_BF16);
  z.out_stride = out_width;
  const int64_t tiles = forward_tiles(num_rows, kTileQ, out_width, kTileP, experts);
  return with_float_type(out_dtype, [&](auto zero) {
    using O = decltype(zero);
    z.out_vectors = rows_fit(out, out_width, out_width, sizeof(O), 16 / (int)sizeof(O));
    return turned ? run<kForwardTurned, O>(maps, offsets, z, out, sms, tiles, stream)
                  : run<kForward, O>(maps, offsets, z, out, sms, tiles, stream);
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
      (out_width > 1 && out_stride < width) || (rc == SEGTOPK_SUCCESS && experts > 1 && expert_stride < width * out_width) || scale_stride < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  const int64_t line = out_width > 1 ? out_stride : width;
  if (experts == 1)
    expert_stride = line;
  if (rc != SEGTOPK_SUCCESS || !float_type_of(out_dtype) || width % 16 != 0 || row_stride > kMaxStride ||
      line > kMaxStride || expert_stride > kMaxStride || forward_tiles(num_rows, kTileP, out_width, kTileP, experts) > kMaxTiles)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  if (num_rows == 0)
    return SEGTOPK_SUCCESS;
  if (!rows || !row_scales || !weights || !weight_scales || !offsets || !out)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!tma_fits(rows, row_stride, 1) || !tma_fits(weights, line, 1) || expert_stride % 16 != 0 ||
      !aligned(offsets, 8) || !aligned(row_scales, 4) || !aligned(weight_scales, 4) ||
      !aligned(out, out_dtype == SEGTOPK_F32 ? 4 : 2))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  Maps maps;
  cudaError_t e = describe(&maps.p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, width, num_rows, 1, row_stride,
                           row_stride, kBox);
  if (e == cudaSuccess)
    e = describe(&maps.large, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, width, num_rows, 1, row_stride, row_stride,
                 kTileP);
  if (e == cudaSuccess)
    e = describe(&maps.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, weights, width, out_width, experts, line, expert_stride,
                 kTileP);
  if (e != cudaSuccess)
    return record_cuda_error(e);
  // Tiles of 128 columns where those of 256 would leave SMs idle. Pairs where
  // experts have rows for both blocks: 131072 rows of 128 experts, 4096x2048,
  // 1073 us, 1143 by single blocks. The rows are counted as if all had an
  // expert; the offsets are the device's.
  const int step = forward_tiles(num_rows, kTileP, out_width, kTileQ, experts) < 2 * sms ? kTileP : kTileQ;
  const bool by_pairs = step == kTileQ && num_rows / experts >= 256;
  const int64_t tiles = forward_tiles(num_rows, kTileP, out_width, step, experts);
  Sizes z = {};
  z.num_rows = num_rows;
  z.experts = experts;
  z.q = (int)out_width;
  z.c = (int)width;
  z.instruction = instruction(by_pairs ? kForward8Pair : kForward8, 0);
  z.out_stride = out_width;
  z.row_scales = row_scales;
  z.scale_stride = scale_stride;
  z.weight_scales = weight_scales;
  z.step = step;
  return with_float_type(out_dtype, [&](auto zero) {
    using O = decltype(zero);
    z.out_vectors = rows_fit(out, out_width, out_width, sizeof(O), 16 / (int)sizeof(O));
    return by_pairs ? run<kForward8Pair, O>(maps, offsets, z, out, sms, tiles, stream)
                    : run<kForward8, O>(maps, offsets, z, out, sms, tiles, stream);
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
  WeightsMaps maps;
  cudaError_t e = cudaSuccess;
  auto add = [&](CUtensorMap* map, const void* rows, int64_t width, int64_t stride, int box) {
    if (e == cudaSuccess)
      e = describe(map, map_type(dtype), 2, rows, width, num_rows, 1, stride, stride, box);
  };
  add(&maps.p, b_rows, b_width, b_stride, kDepth);
  add(&maps.q, a_rows, a_width, a_stride, kDepth);
  for (int i = 0; i < kEndBoxes; ++i) {
    add(&maps.p_end[i], b_rows, b_width, b_stride, 8 >> i);
    add(&maps.q_end[i], a_rows, a_width, a_stride, 8 >> i);
  }
  if (e != cudaSuccess)
    return record_cuda_error(e);
  Sizes z = {};
  z.num_rows = num_rows;
  z.experts = experts;
  z.p = (int)b_width;
  z.q = (int)a_width;
  z.instruction = instruction(kWeights, dtype == SEGTOPK_BF16);
  z.out_stride = b_width;
  return with_float_type(out_dtype, [&](auto zero) {
    using O = decltype(zero);
    z.out_vectors = rows_fit(out, b_width, b_width, sizeof(O), 16 / (int)sizeof(O));
    return run<kWeights, O>(maps, offsets, z, out, sms, tiles, stream);
  });
}

extern "C" int segtopk_test_expert_tile(int32_t rows, int32_t index, int32_t* first, int32_t* width)
{
#ifndef SEGTOPK_TEST_HOOKS
  (void)rows;
  (void)index;
  (void)first;
  (void)width;
  return SEGTOPK_ERROR_NOT_SUPPORTED;
#else
  if (rows < 1 || rows > 2147483647 - kTileQ || index < 0 || index >= pieces(rows, kTileQ) || !first || !width)
    return SEGTOPK_ERROR_INVALID_VALUE;
  const TilePart part = even_part(rows, pieces(rows, kTileQ), index);
  *first = part.first;
  *width = part.width;
  return SEGTOPK_SUCCESS;
#endif
}

extern "C" int segtopk_test_free_row(int32_t first, int32_t end, int32_t index, int64_t* row)
{
#ifndef SEGTOPK_TEST_HOOKS
  (void)first;
  (void)end;
  (void)index;
  (void)row;
  return SEGTOPK_ERROR_NOT_SUPPORTED;
#else
  if (first < 0 || end < first || index < 0 || !row)
    return SEGTOPK_ERROR_INVALID_VALUE;
  *row = free_row(first, end, index);
  return SEGTOPK_SUCCESS;
#endif
}
