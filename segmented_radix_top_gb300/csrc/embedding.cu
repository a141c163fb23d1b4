// Token embedding (segtopk_embedding and segtopk_embedding_backward in
// include/segtopk.h).
//
//   forward   out[i] = c table[token_i]
//   backward  grad_table[v] (+)= c sum over i with token_i = v of grad_out[i]
//
// The backward pass adds each table row's gradients in the order of the
// tokens, without atomics, so that its result does not change from run to
// run: the token positions are sorted by token with a stable radix sort, and
// the sorted positions and the table's rows are merged, each row following
// its positions. Equal shares of that merge go to the groups of threads,
// whatever the tokens' frequencies are. A row whose positions are spread over
// several shares is put together from the shares' 32-bit parts by a last
// kernel.
#include "rank_sort.cuh"

namespace segtopk {
namespace {
using namespace rows;

constexpr int kThreads = 256;
// Of a GB300. Shares and clearing blocks are planned for this number, as the
// workspace's size is, which is asked for without a device; another number of
// SMs would only leave the last wave of blocks less full.
constexpr int kSms = 152;
constexpr int kInFlight = 4; // vectors of a row that a thread has in flight
constexpr int kDigitBits = 9; // of a radix pass: 512 counters a warp in shared memory

template <class I>
__device__ __forceinline__ int64_t row_of_token(const I* tokens, uint32_t i, int64_t vocab)
{
  const int64_t v = (int64_t)tokens[i];
  if (v >= vocab)
    raise_error(SEGTOPK_DEVICE_ERROR_INDEX);
  return v >= 0 && v < vocab ? v : -1;
}

// ---------------------------------------------------------------------------
// Forward: a group of `lanes` threads copies a row
// ---------------------------------------------------------------------------
// Bound by memory with kInFlight vectors a thread under way: 65536 rows of
// 4096 in bf16 114 us, 103 at the copy rate (142 with one vector).
template <class T, class O, int N, class I>
__global__ void __launch_bounds__(kThreads)
lookup_kernel(const T* table, int64_t stride, int64_t vocab, const I* tokens, uint32_t n, int64_t width, int lanes,
              float scale, O* out)
{
  wait_for_previous();
  allow_next();
  const int lane = threadIdx.x & (lanes - 1);
  const uint32_t i = blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  if (i >= n)
    return;
  const int64_t v = row_of_token(tokens, i, vocab);
  constexpr int U = kInFlight;
  const int64_t step = (int64_t)lanes * kPart<N>;
  table += v * stride;
  out += (int64_t)i * width;
  for (int64_t c0 = part_start<N>(lane); c0 < width; c0 += U * step) {
    Part<T, N> got[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v >= 0 && c0 + u * step < width)
        got[u] = load_part<T, N>(table + c0 + u * step, lanes, width - c0 - u * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[kPart<N>];
#pragma unroll
      for (int e = 0; e < kPart<N>; ++e)
        y[e] = v >= 0 ? scale * got[u].f32(e) : 0.0f;
      if (c0 + u * step < width)
        store_part<O, N>(out + c0 + u * step, y, lanes, width - c0 - u * step);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: sort of the positions by token
// ---------------------------------------------------------------------------
// Tokens outside the table, and the padding token, get the key `vocab`, past
// every row.
template <class I>
struct TokenSource {
  const I* tokens;
  int64_t vocab, padding;
  __device__ __forceinline__ uint32_t key(uint32_t i) const
  {
    const int64_t v = row_of_token(tokens, i, vocab);
    return v < 0 || v == padding ? (uint32_t)vocab : (uint32_t)v;
  }
  __device__ __forceinline__ uint32_t at(uint32_t i) const { return i; }
};

// Clears the table while the sort, launched before it, still runs: the sort's
// cluster lets the next kernel start once all its blocks have seen the work
// before them complete, and this one waits for the sort only at its end, so
// that the kernel after it finds both done. (The other order would not do: a
// sort launched second would wait for the clearing first.) Bound by the
// writes. 2048 tokens of 32000 rows of 4 KB: 30 us in all, 40 where the merge
// writes every row after the sort (other sizes at its call); 34 with a block for every 16 KB, whose
// first wave then holds the SMs until the sort ends.
constexpr size_t kClearRun = 32 << 10;
__global__ void __launch_bounds__(kThreads) clear_kernel(char* at, size_t bytes)
{
  allow_next();
  // a block clears runs of consecutive memory
  constexpr int U = kClearRun / (kThreads * 16);
  const bool whole = (((size_t)at | bytes) & 15) == 0;
  for (size_t run = (size_t)blockIdx.x * kClearRun; run < bytes; run += (size_t)gridDim.x * kClearRun) {
    if (whole) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const size_t i = run + (size_t)(u * kThreads + threadIdx.x) * 16;
        if (i < bytes)
          *reinterpret_cast<uint4*>(at + i) = uint4{};
      }
    } else {
      const size_t end = min(bytes, run + kClearRun);
      for (size_t i = run + threadIdx.x * 2; i < end; i += kThreads * 2)
        *reinterpret_cast<uint16_t*>(at + i) = 0;
    }
  }
  wait_for_previous();
}

// ---------------------------------------------------------------------------
// Backward: merge of sorted positions and table rows
// ---------------------------------------------------------------------------
struct Merge {
  const uint64_t* items; // sorted
  uint32_t n;
  uint32_t vocab;
  int64_t width;
  uint32_t shares;
  uint32_t reach; // see row_end()
  int lanes;
  float scale;
  float *head, *carry;          // [shares][width]: parts of rows that several shares hold
  int32_t *head_row, *carry_row; // [shares]: their rows, or -1
  __device__ __forceinline__ uint32_t key(uint32_t i) const { return (uint32_t)items[i]; }
  __device__ __forceinline__ int64_t at(uint32_t i) const { return (int64_t)(items[i] >> 32); }
};

// A share's end (a position) moved past the end of the row it falls into, if
// that is among the next m.reach positions (or as many as the group has lanes
// in a warp). Only the rows of frequent tokens are then held by several
// shares. Short shares have a reach of 0: their sizes would differ too much
// (27 positions a share: 33 us as they are, 38 moved by up to 32).
__device__ __forceinline__ uint32_t row_end(const Merge& m, uint32_t a)
{
  if (m.reach == 0)
    return a;
  const uint32_t g = min(m.lanes, 32), lane = threadIdx.x & 31, mine = lane & (g - 1);
  const unsigned mask = (g == 32 ? kAll : ((1u << g) - 1)) << (lane - mine);
  const uint32_t row = a > 0 ? m.key(a - 1) : 0;
  const bool other = mine <= m.reach && (a + mine >= m.n || m.key(a + mine) != row);
  const unsigned found = __ballot_sync(mask, other) >> (lane - mine);
  return a > 0 && found != 0 ? a + __ffs(found) - 1 : a;
}

// What becomes of the table:
enum Mode {
  kDense, // all rows are written, those without tokens as zeros; a share is a part of the positions and rows together
  kAdd,   // the tokens' rows are added to; a share is a part of the positions
  kWrite  // the tokens' rows are written, the others hold zeros already; shares as for kAdd
};

// The number of positions among the first d[i] steps of the merge, in which
// position a comes before the end of row r if its key is at most r, for both
// ends of a share. The group's lanes (those of a warp at most) try as many places a
// round, so a search takes two or three dependent loads instead of a dozen.
__device__ __forceinline__ void positions_before(const Merge& m, const uint64_t (&d)[2], uint32_t (&a)[2])
{
  const uint32_t g = min(m.lanes, 32), lane = threadIdx.x & 31, mine = lane & (g - 1);
  const unsigned mask = (g == 32 ? kAll : ((1u << g) - 1)) << (lane - mine);
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    lo[i] = (uint32_t)(d[i] > m.vocab ? d[i] - m.vocab : 0);
    hi[i] = (uint32_t)(d[i] < m.n ? d[i] : m.n);
  }
  while (lo[0] < hi[0] || lo[1] < hi[1]) {
    uint32_t at[2];
    bool less[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t span = hi[i] - lo[i];
      // `mine`-th of g places, all different while there are so many
      at[i] = lo[i] + (span <= g ? mine : (uint32_t)((uint64_t)span * (mine + 1) / (g + 1)));
      less[i] = at[i] < hi[i] && (uint64_t)m.key(at[i]) + at[i] < d[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t span = hi[i] - lo[i];
      const uint32_t n = __popc(__ballot_sync(mask, less[i]));
      if (span <= g) {
        lo[i] = hi[i] = lo[i] + n;
      } else {
        const uint32_t low = lo[i];
        if (n > 0)
          lo[i] = low + (uint32_t)((uint64_t)span * n / (g + 1)) + 1;
        if (n < g)
          hi[i] = low + (uint32_t)((uint64_t)span * (n + 1) / (g + 1));
      }
    }
  }
  a[0] = lo[0];
  a[1] = lo[1];
}

// A row is written by the share that holds its last position; if that share
// does not hold the row's first one too, its part goes to `head`, and the
// parts of the shares before it to their `carry`.
//
// Bound by the latency of the gathered rows unless enough of them are under
// way: every thread copies its part of the next kAhead positions' rows (and,
// when adding, of the table rows that they complete) into shared memory of
// its own with asynchronous copies, which takes no registers and, as no
// thread reads another's part, no barrier. 65536 tokens of a table of 152064
// rows of 4096 in bf16: about 270 us for 1.8 GB (262 at the copy rate), 312
// with four rows under way in registers. Elements too badly aligned for
// that (N = 1) go in batches through registers.
template <class G, class W, int N, Mode MODE>
struct Ring {
  static constexpr bool kUsed = N > 1;
  static constexpr int kGrad = N * (int)sizeof(G), kRow = MODE == kAdd ? N * (int)sizeof(W) : 0; // bytes of a position
  static constexpr int kFit = kRingBytes / (kThreads * (kGrad + kRow));
  static constexpr int kAhead = kFit < 16 ? kFit : 16;
  static constexpr int kBytes = kUsed ? kAhead * kThreads * (kGrad + kRow) : 0;
  char* memory;
  __device__ __forceinline__ char* grad(int slot) const { return memory + (slot * kThreads + threadIdx.x) * kGrad; }
  __device__ __forceinline__ char* row(int slot) const
  {
    return memory + kAhead * kThreads * kGrad + (slot * kThreads + threadIdx.x) * kRow;
  }
};

template <class G, class W, int N, Mode MODE>
__global__ void __launch_bounds__(kThreads, N > 1 ? 4 : 3)
merge_kernel(Merge m, const G* grad, int64_t stride, W* out)
{
  wait_for_previous();
  allow_next();
  const int lane = threadIdx.x & (m.lanes - 1);
  const uint32_t p = blockIdx.x * (kThreads / m.lanes) + threadIdx.x / m.lanes;
  constexpr int P = kPart<N>;
  const int64_t c = (int64_t)blockIdx.y * m.lanes * P + part_start<N>(lane), left = m.width - c;
  if (p >= m.shares)
    return;
  const uint64_t steps = (uint64_t)m.n + (MODE == kDense ? m.vocab : 0);
  const uint64_t d[2] = {steps * p / m.shares, steps * (p + 1) / m.shares};
  uint32_t a[2] = {(uint32_t)d[0], (uint32_t)d[1]};
  if (MODE == kDense)
    positions_before(m, d, a);
  const uint32_t a0 = row_end(m, a[0]), a1 = row_end(m, a[1]); // the share's positions
  if (N > 1 && c >= m.width)
    return; // loose elements are guarded one by one
  W* const table = out;
  out += c;
  const uint32_t before = a0 > 0 ? m.key(a0 - 1) : m.vocab;
  bool begun = a0 < a1 && m.key(a0) == before; // the first position's row, by an earlier share
  uint32_t empty = 0;                           // kDense: the next row that may have no position
  if (MODE == kDense) {
    empty = (uint32_t)(d[0] - a[0]);
    empty += empty == before;
  }
  auto clear_to = [&](uint32_t row) {
    if constexpr (N > 1) {
      W* to = out + (int64_t)empty * m.width;
      const Vec<W, N> zero = {};
#pragma unroll 4
      for (; empty < row; ++empty, to += m.width)
        store<W, N>(to, zero);
    } else if (empty < row) {
      // the rows are one run of memory: whole 16 bytes of it, whatever the
      // width, a part for each of the blocks that share its columns
      const int64_t all = (int64_t)(row - empty) * m.width;
      W* from = table + (int64_t)empty * m.width + all * blockIdx.y / gridDim.y;
      W* const to = table + (int64_t)empty * m.width + all * (blockIdx.y + 1) / gridDim.y;
      const int64_t edge = min((int64_t)((16 - ((uintptr_t)from & 15)) & 15) / (int64_t)sizeof(W), to - from);
      for (int64_t e = lane; e < edge; e += m.lanes)
        from[e] = from_f32<W>(0.0f);
      from += edge;
      const int64_t whole = (to - from) * (int64_t)sizeof(W) / 16;
#pragma unroll 4
      for (int64_t v = lane; v < whole; v += m.lanes)
        reinterpret_cast<uint4*>(from)[v] = uint4{};
      for (W* e = from + whole * 16 / (int64_t)sizeof(W) + lane; e < to; e += m.lanes)
        *e = from_f32<W>(0.0f);
    }
    empty = row + 1;
  };

  float acc[P] = {};
  int32_t head_row = -1, carry_row = -1;
  // one position: its key, the next one's, its gradient, and the row it adds
  // to if the keys differ
  auto take = [&](uint32_t key, uint32_t next, const Part<G, N>& v, const Part<W, N>& was) {
    if (MODE == kDense)
      clear_to(key);
#pragma unroll
    for (int e = 0; e < P; ++e)
      acc[e] += v.f32(e);
    carry_row = (int32_t)key;
    if (next == key)
      return;
    if (begun) {
      store_part<float, N>(m.head + (int64_t)p * m.width + c, acc, m.lanes, left);
      head_row = carry_row;
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e)
        acc[e] = MODE == kAdd ? fmaf(m.scale, acc[e], was.f32(e)) : m.scale * acc[e];
      store_part<W, N>(out + (int64_t)key * m.width, acc, m.lanes, left);
    }
    begun = false;
    carry_row = -1;
#pragma unroll
    for (int e = 0; e < P; ++e)
      acc[e] = 0;
  };
  auto key_at = [&](uint32_t i) { return i < m.n ? m.key(i) : m.vocab; };
  grad += c;

  using R = Ring<G, W, N, MODE>;
  if constexpr (R::kUsed) {
    extern __shared__ uint4 ring_memory[];
    const R ring = {reinterpret_cast<char*>(ring_memory)};
    constexpr int A = R::kAhead;
    uint32_t ahead = key_at(a0); // key of the next position to copy
    auto copy = [&](uint32_t i, int slot) {
      if (i < a1) {
        const uint32_t key = ahead;
        ahead = key_at(i + 1);
        if (key < m.vocab) {
          copy_async<R::kGrad>(ring.grad(slot), grad + m.at(i) * stride);
          if constexpr (MODE == kAdd)
            if (ahead != key)
              copy_async<R::kRow>(ring.row(slot), out + (int64_t)key * m.width);
        }
      }
      commit_copies(); // a group for every position, empty past the end
    };
    for (int u = 0; u < A; ++u)
      copy(a0 + u, u);
    uint32_t key = key_at(a0);
    int slot = 0;
    for (uint32_t i = a0; i < a1; ++i) {
      const uint32_t next = key_at(i + 1);
      wait_for_copies<A - 1>();
      if (key < m.vocab) {
        Vec<W, N> was = {};
        if constexpr (MODE == kAdd)
          was = load<W, N>(reinterpret_cast<const W*>(ring.row(slot)));
        take(key, next, load<G, N>(reinterpret_cast<const G*>(ring.grad(slot))), was);
      }
      copy(i + A, slot);
      slot = slot + 1 == A ? 0 : slot + 1;
      key = next;
    }
  } else {
    constexpr int U = MODE == kAdd ? 4 : 8;
    for (uint32_t i = a0; i < a1; i += U) {
      uint32_t key[U + 1]; // vocab: none
      Part<G, N> v[U];
      Part<W, N> was[U];
#pragma unroll
      for (int u = 0; u <= U; ++u)
        key[u] = key_at(i + u);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u < a1 && key[u] < m.vocab)
          v[u] = load_part<G, N>(grad + m.at(i + u) * stride, m.lanes, left);
        if (MODE == kAdd && i + u < a1 && key[u] < m.vocab && key[u + 1] != key[u])
          was[u] = load_part<W, N>(out + (int64_t)key[u] * m.width, m.lanes, left);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u < a1 && key[u] < m.vocab)
          take(key[u], key[u + 1], v[u], was[u]);
    }
  }
  if (MODE == kDense)
    clear_to((uint32_t)(d[1] - a[1]));
  if (carry_row >= 0)
    store_part<float, N>(m.carry + (int64_t)p * m.width + c, acc, m.lanes, left);
  if (c == 0) {
    m.head_row[p] = head_row;
    m.carry_row[p] = carry_row;
  }
}

// A row that began in shares before p and ended in p: the parts that those
// left, in their order, and p's own. A block looks at one share or several
// and serves kJoinCols columns, a thread four of them. The row of a frequent
// token has parts in many shares: from kJoinSplit on, each warp sums a run of
// them over all the block's columns, and the runs' sums are added in order.
// About 5 us in a stream: the latency of finding and adding the longest run.
constexpr uint32_t kJoinShares = 8; // where most have no such row, else one
constexpr int kJoinCols = kThreads * 4;
constexpr uint32_t kJoinSplit = 48;

template <class W, int N, Mode MODE>
__device__ __forceinline__ void join_row(const Merge& m, uint32_t p, int32_t row, W* out,
                                         float (*part)[kJoinCols])
{
  constexpr int kWarps = kThreads / 32;
  constexpr int kTiles = kJoinCols / (32 * N); // a warp's accesses for the block's columns
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t first = p; // of the shares that hold a part
  for (bool more = true; more;) {
    const bool held = first > (uint32_t)lane && m.carry_row[first - 1 - lane] == row;
    const uint32_t n = __ffs(~__ballot_sync(kAll, held)) - 1u; // all ones: none, so -1
    more = n > 31;
    first -= more ? 32 : n;
  }
  const int64_t c0 = (int64_t)blockIdx.y * kJoinCols;
  const int cols = (int)min((int64_t)kJoinCols, m.width - c0);
  const float* carry = m.carry + c0;
  auto write = [&](int c, const float (&sum)[N]) {
    const Vec<float, N> v = load<float, N>(m.head + (int64_t)p * m.width + c0 + c);
    W* to = out + (int64_t)row * m.width + c0 + c;
    Vec<W, N> was = {};
    if constexpr (MODE == kAdd)
      was = load<W, N>(to);
    float y[N];
#pragma unroll
    for (int e = 0; e < N; ++e)
      y[e] = MODE == kAdd ? fmaf(m.scale, sum[e] + v.f32(e), was.f32(e)) : m.scale * (sum[e] + v.f32(e));
    store_f32<W, N>(to, y);
  };

  const uint32_t parts = p - first;
  if (parts < kJoinSplit) {
    for (int c = threadIdx.x * N; c < cols; c += kThreads * N) {
      float sum[N] = {};
#pragma unroll 8
      for (uint32_t q = first; q < p; ++q) {
        const Vec<float, N> v = load<float, N>(carry + (int64_t)q * m.width + c);
#pragma unroll
        for (int e = 0; e < N; ++e)
          sum[e] += v.f32(e);
      }
      write(c, sum);
    }
    return;
  }
  const uint32_t q0 = first + (uint32_t)((uint64_t)parts * warp / kWarps);
  const uint32_t q1 = first + (uint32_t)((uint64_t)parts * (warp + 1) / kWarps);
  constexpr int kAtOnce = kTiles < 8 ? kTiles : 8;
  for (int t0 = 0; t0 < kTiles; t0 += kAtOnce) {
    float sum[kAtOnce][N] = {};
#pragma unroll 2
    for (uint32_t q = q0; q < q1; ++q) {
#pragma unroll
      for (int t = 0; t < kAtOnce; ++t) {
        const int c = ((t0 + t) * 32 + lane) * N;
        if (c < cols) {
          const Vec<float, N> v = load<float, N>(carry + (int64_t)q * m.width + c);
#pragma unroll
          for (int e = 0; e < N; ++e)
            sum[t][e] += v.f32(e);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kAtOnce; ++t)
#pragma unroll
      for (int e = 0; e < N; ++e)
        part[warp][((t0 + t) * 32 + lane) * N + e] = sum[t][e];
  }
  __syncthreads();
  for (int c = threadIdx.x * N; c < cols; c += kThreads * N) {
    float sum[N] = {};
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int e = 0; e < N; ++e)
        sum[e] += part[w][c + e];
    write(c, sum);
  }
}

template <class W, int N, Mode MODE>
__global__ void __launch_bounds__(kThreads) join_kernel(Merge m, W* out)
{
  __shared__ float part[kThreads / 32][kJoinCols];
  wait_for_previous();
  allow_next();
  const uint32_t count = m.reach > 0 ? kJoinShares : 1;
  const uint32_t first = blockIdx.x * count, lane = threadIdx.x & 31;
  const bool mine = lane < count && first + lane < m.shares;
  const int32_t row = mine ? m.head_row[first + lane] : -1; // every warp the same ones
  for (unsigned left = __ballot_sync(kAll, row >= 0); left != 0; left &= left - 1) {
    const int i = __ffs(left) - 1;
    join_row<W, N, MODE>(m, first + i, __shfl_sync(kAll, row, i), out, part);
    __syncthreads(); // part is written again
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct Layout {
  SortPlan sort;
  uint32_t most_shares;                         // of any call with these sizes
  size_t items, copy, counts, parts, rows, total; // bytes of each piece
};

// Shares of the merge where a row takes row_threads threads: as many groups as
// are resident, or a multiple of that where every share then still has 32
// steps (each costs a search and up to two parts of rows), so that the last
// wave of blocks is a full one; never less than eight steps a share.
uint32_t shares_of(int64_t steps, int64_t row_threads)
{
  const int64_t resident = std::max<int64_t>(1, kSms * 1024 / std::max<int64_t>(1, row_threads));
  const int64_t waves = std::min<int64_t>(9, std::max<int64_t>(1, steps / (32 * resident)));
  return (uint32_t)std::max<int64_t>(1, std::min<int64_t>(resident * waves, (steps + 7) / 8));
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

Layout layout_of(int64_t n, int64_t vocab, int64_t width)
{
  Layout l;
  int bits = 1;
  while ((vocab >> bits) != 0) // keys are 0 .. vocab
    ++bits;
  const int passes = (bits + kDigitBits - 1) / kDigitBits, digit_bits = (bits + passes - 1) / passes;
  l.sort = sort_plan(n, passes, digit_bits, 1 << digit_bits);
  l.most_shares = shares_of(n + vocab, (width + 7) / 8); // eight columns a thread: the fewest threads
  l.items = round_up((size_t)n * 8);
  l.copy = round_up(l.sort.copy());
  l.counts = round_up(l.sort.counts());
  l.parts = round_up((size_t)l.most_shares * (size_t)width * 4);
  l.rows = round_up((size_t)l.most_shares * 4);
  l.total = l.items + 2 * l.copy + l.counts + 2 * l.parts + 2 * l.rows;
  return l;
}

constexpr size_t kClearBlocks = 7 * kSms;
constexpr int64_t kFewOf = 4; // tokens are few of a table's rows if not more than one in as many
constexpr int64_t kMaxVocab = 2147483646LL;
bool fits(int64_t n, int64_t vocab, int64_t width)
{
  return n >= 0 && n <= 2147483647LL && vocab >= 1 && vocab <= kMaxVocab && width >= 0 && width <= (1 << 20);
}

} // namespace

cudaError_t read_embedding_error(uint32_t* word)
{
  const uint32_t zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(word, g_device_error, sizeof(zero));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
}

} // namespace segtopk

using namespace segtopk;

extern "C" int segtopk_embedding(segtopk_dtype dtype, const void* table, int64_t vocab, int64_t width,
                                 int64_t row_stride, const void* tokens, int32_t token_bytes, int64_t num_tokens,
                                 float scale, segtopk_dtype out_dtype, void* out, void* stream)
{
  record_launch_count(0);
  if ((token_bytes != 4 && token_bytes != 8) || num_tokens < 0 || vocab < 1 || width < 0 ||
      row_stride < 0 || dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 || out_dtype < SEGTOPK_F16 ||
      out_dtype > SEGTOPK_I32)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!fits(num_tokens, vocab, width))
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  return with_float_type(dtype, [&](auto zero_in) {
    return with_float_type(out_dtype, [&](auto zero_out) {
      using T = decltype(zero_in);
      using O = decltype(zero_out);
      constexpr int N = 16 / (int)sizeof(T);
      if (num_tokens == 0 || width == 0)
        return (int)SEGTOPK_SUCCESS;
      if (!table || !tokens || !out)
        return (int)SEGTOPK_ERROR_INVALID_VALUE;
      if (!aligned(table, sizeof(T)) || !aligned(out, sizeof(O)) || !aligned(tokens, token_bytes))
        return (int)SEGTOPK_ERROR_MISALIGNED;
      int sms;
      const int bad = check_device(&sms);
      if (bad != SEGTOPK_SUCCESS)
        return bad;
      auto go = [&](auto n, auto id) {
        constexpr int V = decltype(n)::value;
        using I = decltype(id);
        const int lanes = lanes_for((parts_of(width, V) + kInFlight - 1) / kInFlight, kThreads);
        const int64_t per_block = kThreads / lanes;
        return finish(launch(lookup_kernel<T, O, V, I>, dim3((unsigned)((num_tokens + per_block - 1) / per_block)),
                             kThreads, 0, (cudaStream_t)stream, (const T*)table, row_stride, vocab, (const I*)tokens,
                             (uint32_t)num_tokens, width, lanes, scale, (O*)out), 1);
      };
      const bool vector = rows_fit(table, row_stride, width, sizeof(T), N) && rows_fit(out, width, width, sizeof(O), N);
      auto by_id = [&](auto id) {
        return vector ? go(std::integral_constant<int, N>{}, id) : go(std::integral_constant<int, 1>{}, id);
      };
      return token_bytes == 4 ? by_id(int32_t{}) : by_id(int64_t{});
    });
  });
}

extern "C" size_t segtopk_embedding_backward_workspace_bytes(int64_t num_tokens, int64_t vocab, int64_t width)
{
  return fits(num_tokens, vocab, width) ? layout_of(num_tokens, vocab, width).total : 0;
}

extern "C" int segtopk_embedding_backward(segtopk_dtype dtype, const void* grad_out, int64_t grad_stride,
                                          const void* tokens, int32_t token_bytes, int64_t num_tokens, int64_t vocab,
                                          int64_t width, int64_t padding_token, float scale,
                                          segtopk_dtype table_dtype, void* grad_table, int accumulate,
                                          void* workspace, size_t workspace_bytes, void* stream)
{
  record_launch_count(0);
  if ((token_bytes != 4 && token_bytes != 8) || num_tokens < 0 || vocab < 1 || width < 0 ||
      grad_stride < 0 || dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 ||
      table_dtype < SEGTOPK_F16 || table_dtype > SEGTOPK_I32 || (accumulate != 0 && accumulate != 1))
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!fits(num_tokens, vocab, width))
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  return with_float_type(dtype, [&](auto zero_in) {
    return with_float_type(table_dtype, [&](auto zero_out) {
      using G = decltype(zero_in);
      using W = decltype(zero_out);
      constexpr int N = 16 / (int)std::max(sizeof(G), sizeof(W)); // no access above 16 bytes
      if (width == 0 || (accumulate && num_tokens == 0))
        return (int)SEGTOPK_SUCCESS;
      if ((num_tokens > 0 && (!grad_out || !tokens)) || !grad_table)
        return (int)SEGTOPK_ERROR_INVALID_VALUE;
      if (!aligned(grad_out, sizeof(G)) || !aligned(grad_table, sizeof(W)) || !aligned(tokens, token_bytes) ||
          !aligned(workspace, 256))
        return (int)SEGTOPK_ERROR_MISALIGNED;
      const Layout l = layout_of(num_tokens, vocab, width);
      if (!workspace || workspace_bytes < l.total)
        return (int)SEGTOPK_ERROR_INVALID_VALUE;
      int sms;
      const int bad = check_device(&sms);
      if (bad != SEGTOPK_SUCCESS)
        return bad;
      char* w = (char*)workspace;
      auto piece = [&](size_t bytes) {
        char* at = w;
        w += bytes;
        return at;
      };
      uint64_t* items = (uint64_t*)piece(l.items);
      uint64_t* const copies[2] = {(uint64_t*)piece(l.copy), (uint64_t*)piece(l.copy)};
      uint32_t* counts = (uint32_t*)piece(l.counts);
      cudaStream_t st = (cudaStream_t)stream;
      cudaError_t e = cudaSuccess;
      const uint32_t n = (uint32_t)num_tokens;
      // Clearing the table beside the sort, on the SMs that a cluster leaves,
      // and then writing the tokens' rows writes those twice: worth it where
      // they are few of all. 32000 rows of 4 KB, ids with a text's frequencies:
      // 2048 tokens 30 against 40 us, 4096 33 against 44, 8000 37 against 48;
      // uniform ids 29 against 38, 32 against 42, 36 against 44. The two meet
      // above a quarter (at 8192 the step is still 36 to 44).
      const bool clear_first = !accumulate && l.sort.tiles.items == 0 && num_tokens <= vocab / kFewOf;
      int launches = 0;
      if (n > 0 || clear_first) { // the clearing follows a sort, of no tokens too
        auto by = [&](auto id) {
          using I = decltype(id);
          return sort<false>(l.sort, TokenSource<I>{(const I*)tokens, vocab, padding_token}, ItemSink{items}, copies,
                             counts, st, &e);
        };
        launches = token_bytes == 4 ? by(int32_t{}) : by(int64_t{});
        if (launches < 0)
          return record_cuda_error(e);
      }
      if (clear_first) {
        const size_t bytes = (size_t)vocab * (size_t)width * sizeof(W);
        // fewer blocks than fill the SMs: one that has cleared its runs stays
        // until the sort is done, and the merge's blocks come in beside them
        const unsigned blocks = (unsigned)std::min<size_t>(kClearBlocks, (bytes + kClearRun - 1) / kClearRun);
        e = launch(clear_kernel, dim3(blocks), kThreads, 0, st, (char*)grad_table, bytes);
        if (e != cudaSuccess)
          return record_cuda_error(e);
        ++launches;
      }
      if (clear_first && n == 0)
        return finish(e, launches);
      auto go = [&](auto nv, auto mode) {
        constexpr int V = decltype(nv)::value;
        constexpr Mode MODE = decltype(mode)::value;
        Merge m = {};
        m.items = items;
        m.n = n;
        m.vocab = (uint32_t)vocab;
        m.width = width;
        // no share without a step: a row's shares have to be neighbours
        m.lanes = lanes_for(parts_of(width, V), kThreads);
        const int64_t cols = (int64_t)m.lanes * (V > 1 ? V : kLoose), tiles = (width + cols - 1) / cols;
        m.shares = std::min(l.most_shares, shares_of((int64_t)n + (MODE == kDense ? vocab : 0), m.lanes * tiles));
        const uint32_t a_share = (uint32_t)(((int64_t)n + (MODE == kDense ? vocab : 0)) / m.shares);
        m.reach = a_share >= 64 ? std::min(32u, a_share / 4) : 0;
        m.scale = scale;
        m.head = (float*)piece(l.parts);
        m.carry = (float*)piece(l.parts);
        m.head_row = (int32_t*)piece(l.rows);
        m.carry_row = (int32_t*)piece(l.rows);
        const uint32_t per_block = (uint32_t)(kThreads / m.lanes);
        const dim3 grid((m.shares + per_block - 1) / per_block, (unsigned)tiles);
        e = launch(merge_kernel<G, W, V, MODE>, grid, kThreads, Ring<G, W, V, MODE>::kBytes, st, m,
                   (const G*)grad_out, grad_stride, (W*)grad_table);
        constexpr int J = V > 4 ? 4 : V; // columns of a thread: 16 bytes of the parts
        const uint32_t looks = m.reach > 0 ? kJoinShares : 1; // of a block: see join_kernel
        const dim3 joins((m.shares + looks - 1) / looks, (unsigned)((width + kJoinCols - 1) / kJoinCols));
        if (e == cudaSuccess)
          e = launch(join_kernel<W, J, MODE>, joins, kThreads, 0, st, m, (W*)grad_table);
        return finish(e, launches + 2);
      };
      const bool vector = rows_fit(grad_out, grad_stride, width, sizeof(G), N) &&
                          rows_fit(grad_table, width, width, sizeof(W), N);
      using One = std::integral_constant<int, 1>;
      using Many = std::integral_constant<int, N>;
      auto by_mode = [&](auto mode) { return vector ? go(Many{}, mode) : go(One{}, mode); };
      if (accumulate)
        return by_mode(std::integral_constant<Mode, kAdd>{});
      return clear_first ? by_mode(std::integral_constant<Mode, kWrite>{}) : by_mode(std::integral_constant<Mode, kDense>{});
    });
  });
}
