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
constexpr int kSms = 152;
constexpr int kInFlight = 4; // vectors of a row that a thread has in flight
constexpr int kDigitBits = 9; // of a radix pass: 512 counters a warp in shared memory

__device__ uint32_t g_error;

template <class I>
__device__ __forceinline__ int64_t row_of_token(const I* tokens, uint32_t i, int64_t vocab)
{
  const int64_t v = (int64_t)*(tokens + i);
  if (v >= vocab)
    atomicOr(&g_error, (uint32_t)SEGTOPK_DEVICE_ERROR_INDEX);
  return v >= 0 && v < vocab ? v : -1;
}

// ---------------------------------------------------------------------------
// Forward: a group of `lanes` threads copies a row
// ---------------------------------------------------------------------------
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
  const int64_t step = (int64_t)lanes * N;
  for (int64_t c0 = (int64_t)lane * N; c0 < width; c0 += U * step) {
    Vec<T, N> got[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v >= 0 && c0 + u * step < width)
        got[u] = load<T, N>(table + v * stride + c0 + u * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[N];
#pragma unroll
      for (int e = 0; e < N; ++e)
        y[e] = v >= 0 ? scale * got[u].f32(e) : 0.0f;
      if (c0 + u * step < width)
        store_f32<O, N>(out + (int64_t)i * width + c0 + u * step, y);
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
  uint32_t mask;
  struct Item {
    uint32_t digit, key, at;
  };
  __device__ __forceinline__ uint32_t key(uint32_t i) const
  {
    const int64_t v = row_of_token(tokens, i, vocab);
    return v < 0 || v == padding ? (uint32_t)vocab : (uint32_t)v;
  }
  __device__ __forceinline__ uint32_t digit(uint32_t i) const { return key(i) & mask; }
  __device__ __forceinline__ Item load(uint32_t i) const
  {
    const uint32_t k = key(i);
    return {k & mask, k, i};
  }
};
struct PairSource {
  const uint32_t *keys, *at;
  int shift;
  uint32_t mask;
  struct Item {
    uint32_t digit, key, at;
  };
  __device__ __forceinline__ uint32_t digit(uint32_t i) const { return (keys[i] >> shift) & mask; }
  __device__ __forceinline__ Item load(uint32_t i) const { return {digit(i), keys[i], at[i]}; }
};
struct PairSink {
  uint32_t *keys, *at;
  template <class Item>
  __device__ __forceinline__ void put(uint32_t, Item item, uint32_t place) const
  {
    keys[place] = item.key;
    at[place] = item.at;
  }
  __device__ __forceinline__ void start(int, uint32_t) const {}
};

// ---------------------------------------------------------------------------
// Backward: merge of sorted positions and table rows
// ---------------------------------------------------------------------------
struct Merge {
  const uint32_t *keys, *at; // sorted
  uint32_t n;
  uint32_t vocab;
  int64_t width;
  uint32_t shares;
  int lanes;
  float scale;
  float *head, *carry;          // [shares][width]: parts of rows that several shares hold
  int32_t *head_row, *carry_row; // [shares]: their rows, or -1
};

// The number of positions among the first d[i] steps of the merge, in which
// position a comes before the end of row r if keys[a] <= r, for both ends of
// a share. The group's lanes (those of a warp at most) try as many places a
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
      less[i] = at[i] < hi[i] && (uint64_t)m.keys[at[i]] + at[i] < d[i];
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

// DENSE: every row of the table is written, rows without tokens as zeros, and
// a share is a part of the positions and rows together. Otherwise only the
// tokens' rows are added to, and a share is a part of the positions.
template <class G, class W, int N, bool DENSE>
__global__ void __launch_bounds__(kThreads)
merge_kernel(Merge m, const G* grad, int64_t stride, W* out)
{
  wait_for_previous();
  allow_next();
  const int lane = threadIdx.x & (m.lanes - 1);
  const uint32_t p = blockIdx.x * (kThreads / m.lanes) + threadIdx.x / m.lanes;
  const int64_t c = ((int64_t)blockIdx.y * m.lanes + lane) * N;
  if (p >= m.shares)
    return;
  const uint64_t steps = (uint64_t)m.n + (DENSE ? m.vocab : 0);
  const uint64_t d[2] = {steps * p / m.shares, steps * (p + 1) / m.shares};
  uint32_t a[2] = {(uint32_t)d[0], (uint32_t)d[1]};
  if (DENSE)
    positions_before(m, d, a);
  if (c >= m.width)
    return;
  const uint32_t a0 = a[0], a1 = a[1];
  const uint32_t r1 = DENSE ? (uint32_t)(d[1] - a1) : m.vocab;
  uint32_t row = DENSE ? (uint32_t)(d[0] - a0) : (a0 < a1 ? m.keys[a0] : m.vocab);
  bool begun = a0 > 0 && row < m.vocab && m.keys[a0 - 1] == row; // by an earlier share
  bool any = false;
  int32_t head_row = -1, carry_row = -1;
  float acc[N] = {};

  auto finish_row = [&]() {
    if (begun) {
      store_f32<float, N>(m.head + (int64_t)p * m.width + c, acc);
      head_row = (int32_t)row;
      begun = false;
    } else {
      W* to = out + (int64_t)row * m.width + c;
      float y[N];
#pragma unroll
      for (int e = 0; e < N; ++e)
        y[e] = m.scale * acc[e];
      if constexpr (!DENSE) {
        const Vec<W, N> was = load<W, N>(to);
#pragma unroll
        for (int e = 0; e < N; ++e)
          y[e] += was.f32(e);
      }
      store_f32<W, N>(to, y);
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
      acc[e] = 0;
    any = false;
  };

  constexpr int U = 4; // rows in flight
  for (uint32_t i = a0; i < a1; i += U) {
    uint32_t key[U];
    Vec<G, N> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      key[u] = i + u < a1 ? m.keys[i + u] : m.vocab;
      if (key[u] < m.vocab)
        v[u] = load<G, N>(grad + (int64_t)m.at[i + u] * stride + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (key[u] >= m.vocab)
        continue;
      if (DENSE) {
        for (; row < key[u]; ++row)
          finish_row();
      } else if (row != key[u]) {
        finish_row();
        row = key[u];
      }
#pragma unroll
      for (int e = 0; e < N; ++e)
        acc[e] += v[u].f32(e);
      any = true;
    }
  }
  if (DENSE) {
    for (; row < r1; ++row)
      finish_row();
  } else if (any && !(a1 < m.n && m.keys[a1] == row)) {
    finish_row();
  }
  if (any) {
    store_f32<float, N>(m.carry + (int64_t)p * m.width + c, acc);
    carry_row = (int32_t)row;
  }
  if (c == 0) {
    m.head_row[p] = head_row;
    m.carry_row[p] = carry_row;
  }
}

// A row that began in shares before p and ended in p: the parts that those
// left, in their order, and p's own. A block serves one share and kJoinCols
// columns. A frequent token leaves its row's parts in many shares; from
// kJoinSplit parts on the block's warps sum a run of them each, and the runs'
// sums are added in order.
constexpr int kJoinCols = kThreads * 4;
constexpr uint32_t kJoinSplit = 16;

template <class W, int N, bool DENSE>
__global__ void __launch_bounds__(kThreads) join_kernel(Merge m, W* out)
{
  __shared__ float part[kThreads / 32][32 * N];
  wait_for_previous();
  allow_next();
  const uint32_t p = blockIdx.x;
  const int32_t row = m.head_row[p];
  if (row < 0)
    return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t first = p; // of the shares that hold a part
  for (bool more = true; more;) {
    const bool held = first > (uint32_t)lane && m.carry_row[first - 1 - lane] == row;
    const uint32_t n = __ffs(~__ballot_sync(kAll, held)) - 1u; // all ones: none, so -1
    more = n > 31;
    first -= more ? 32 : n;
  }

  auto sum = [&](uint32_t q, uint32_t end, int64_t c, float (&acc)[N]) {
#pragma unroll 4
    for (; q < end; ++q) {
      const Vec<float, N> v = load<float, N>(m.carry + (int64_t)q * m.width + c);
#pragma unroll
      for (int e = 0; e < N; ++e)
        acc[e] += v.f32(e);
    }
  };
  auto write = [&](int64_t c, const float (&acc)[N]) {
    const Vec<float, N> v = load<float, N>(m.head + (int64_t)p * m.width + c);
    W* to = out + (int64_t)row * m.width + c;
    float y[N];
#pragma unroll
    for (int e = 0; e < N; ++e)
      y[e] = m.scale * (acc[e] + v.f32(e));
    if constexpr (!DENSE) {
      const Vec<W, N> was = load<W, N>(to);
#pragma unroll
      for (int e = 0; e < N; ++e)
        y[e] += was.f32(e);
    }
    store_f32<W, N>(to, y);
  };

  const int64_t c0 = (int64_t)blockIdx.y * kJoinCols, c1 = min(m.width, c0 + kJoinCols);
  const uint32_t parts = p - first;
  if (parts < kJoinSplit) {
    for (int64_t c = c0 + (int64_t)threadIdx.x * N; c < c1; c += (int64_t)kThreads * N) {
      float acc[N] = {};
      sum(first, p, c, acc);
      write(c, acc);
    }
    return;
  }
  constexpr uint32_t kWarps = kThreads / 32;
  const uint32_t q0 = first + (uint32_t)((uint64_t)parts * warp / kWarps);
  const uint32_t q1 = first + (uint32_t)((uint64_t)parts * (warp + 1) / kWarps);
  for (int64_t t = c0; t < c1; t += 32 * N) {
    const int64_t c = t + lane * N;
    float acc[N] = {};
    if (c < c1)
      sum(q0, q1, c, acc);
#pragma unroll
    for (int e = 0; e < N; ++e)
      part[warp][lane * N + e] = acc[e];
    __syncthreads();
    if (warp == 0 && c < c1) {
      for (uint32_t w = 1; w < kWarps; ++w)
#pragma unroll
        for (int e = 0; e < N; ++e)
          acc[e] += part[w][lane * N + e];
      write(c, acc);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct Layout {
  int passes, digit_bits;
  Tiling tiles;
  uint32_t most_shares; // of any call with these sizes
  size_t pairs, counts, parts, rows, total; // bytes of each piece
};

// Shares of the merge: at most twice as many groups as are resident, of 16
// steps at least (a share costs a search and up to two parts of rows).
uint32_t shares_of(int64_t steps, int64_t width)
{
  const int64_t most = 2 * (int64_t)kSms * 2048 / std::max<int64_t>(1, std::min<int64_t>((width + 7) / 8, 2048));
  return (uint32_t)std::max<int64_t>(1, std::min<int64_t>(most, (steps + 15) / 16));
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

Layout layout_of(int64_t n, int64_t vocab, int64_t width)
{
  Layout l;
  int bits = 1;
  while ((vocab >> bits) != 0) // keys are 0 .. vocab
    ++bits;
  l.passes = (bits + kDigitBits - 1) / kDigitBits;
  l.digit_bits = (bits + l.passes - 1) / l.passes;
  l.tiles = tiling(n);
  l.most_shares = shares_of(n + vocab, width);
  l.pairs = round_up((size_t)n * 4);
  l.counts = round_up(count_bytes(l.tiles, 1 << l.digit_bits));
  l.parts = round_up((size_t)l.most_shares * (size_t)width * 4);
  l.rows = round_up((size_t)l.most_shares * 4);
  l.total = 4 * l.pairs + l.counts + 2 * l.parts + 2 * l.rows;
  return l;
}

constexpr int64_t kMaxVocab = 2147483646LL;
bool fits(int64_t n, int64_t vocab, int64_t width)
{
  return n >= 0 && n <= 2147483647LL && vocab >= 1 && vocab <= kMaxVocab && width >= 0 && width <= (1 << 20);
}

} // namespace

cudaError_t read_embedding_error(uint32_t* word)
{
  const uint32_t zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(word, g_error, sizeof(zero));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_error, &zero, sizeof(zero));
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
        const int lanes = lanes_for((width / V + kInFlight - 1) / kInFlight, kThreads);
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
      constexpr int N = 16 / (int)sizeof(G);
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
      uint32_t* keys[2] = {(uint32_t*)piece(l.pairs), (uint32_t*)piece(l.pairs)};
      uint32_t* at[2] = {(uint32_t*)piece(l.pairs), (uint32_t*)piece(l.pairs)};
      uint32_t* counts = (uint32_t*)piece(l.counts);
      cudaStream_t st = (cudaStream_t)stream;
      cudaError_t e = cudaSuccess;
      int launches = 0, to = 0;
      const uint32_t n = (uint32_t)num_tokens;
      const int bins = 1 << l.digit_bits;
      for (int pass = 0; pass < l.passes && n > 0; ++pass) {
        const PairSink sink = {keys[to], at[to]};
        int made;
        if (pass > 0)
          made = rank_pass(PairSource{keys[1 - to], at[1 - to], pass * l.digit_bits, (uint32_t)bins - 1}, sink, n,
                           l.tiles, bins, counts, st, &e);
        else if (token_bytes == 4)
          made = rank_pass(TokenSource<int32_t>{(const int32_t*)tokens, vocab, padding_token, (uint32_t)bins - 1},
                           sink, n, l.tiles, bins, counts, st, &e);
        else
          made = rank_pass(TokenSource<int64_t>{(const int64_t*)tokens, vocab, padding_token, (uint32_t)bins - 1},
                           sink, n, l.tiles, bins, counts, st, &e);
        if (made < 0)
          return record_cuda_error(e);
        launches += made;
        to = 1 - to;
      }
      auto go = [&](auto nv, auto all) {
        constexpr int V = decltype(nv)::value;
        constexpr bool DENSE = decltype(all)::value;
        Merge m = {};
        m.keys = keys[1 - to];
        m.at = at[1 - to];
        m.n = n;
        m.vocab = (uint32_t)vocab;
        m.width = width;
        // no share without a step: a row's shares have to be neighbours
        m.shares = shares_of((int64_t)n + (DENSE ? vocab : 0), width);
        m.lanes = lanes_for(width / V, kThreads);
        m.scale = scale;
        m.head = (float*)piece(l.parts);
        m.carry = (float*)piece(l.parts);
        m.head_row = (int32_t*)piece(l.rows);
        m.carry_row = (int32_t*)piece(l.rows);
        const uint32_t per_block = (uint32_t)(kThreads / m.lanes);
        const int64_t cols = (int64_t)m.lanes * V;
        const dim3 grid((m.shares + per_block - 1) / per_block, (unsigned)((width + cols - 1) / cols));
        e = launch(merge_kernel<G, W, V, DENSE>, grid, kThreads, 0, st, m, (const G*)grad_out, grad_stride,
                   (W*)grad_table);
        constexpr int J = V > 4 ? 4 : V; // columns of a thread: 16 bytes of the parts
        const dim3 joins(m.shares, (unsigned)((width + kJoinCols - 1) / kJoinCols));
        if (e == cudaSuccess)
          e = launch(join_kernel<W, J, DENSE>, joins, kThreads, 0, st, m, (W*)grad_table);
        return finish(e, launches + 2);
      };
      const bool vector = rows_fit(grad_out, grad_stride, width, sizeof(G), N) &&
                          rows_fit(grad_table, width, width, sizeof(W), N);
      using One = std::integral_constant<int, 1>;
      using Many = std::integral_constant<int, N>;
      if (accumulate)
        return vector ? go(Many{}, std::false_type{}) : go(One{}, std::false_type{});
      return vector ? go(Many{}, std::true_type{}) : go(One{}, std::true_type{});
    });
  });
}
