// Rows moved to expert order and back (segtopk_dispatch, segtopk_combine and
// segtopk_combine_backward in include/segtopk.h).
//
//   dispatch          rows[r(t, j)] = x[t]
//   combine           out[t] = sum_j w_tj rows[r(t, j)]
//   combine backward  grad_rows[r(t, j)] = w_tj g[t],  grad_w_tj = <rows[r(t, j)], g[t]>
//
// r(t, j) is the row of token t's j-th slot, or none. Every kernel goes by
// token, so a token's row is read or written once and only the k sorted rows
// are scattered; all are bound by memory bandwidth, if the gathered rows are
// asked for early enough. 8192 tokens of 2048 in bf16, k = 8: copy 46 us, sum
// 50, unweighted 51, backward 97 (44, 44, 44 and 84 at the copy rate); 32768
// of 4096: copy and sum 355 each (356).
#include "rows.cuh"

namespace segtopk {
namespace {
using namespace rows;

constexpr int kThreads = 256;

// The row of a slot, or -1: one outside the sorted rows counts as none.
__device__ __forceinline__ int32_t row_at(const int32_t* row_of_slot, uint32_t slots)
{
  const int32_t r = *row_of_slot;
  return (uint32_t)r < slots ? r : -1;
}

// A group of `lanes` threads (a power of two, at most kThreads) serves a
// token.
struct Shape {
  uint32_t tokens;
  int k;
  int64_t width;
  int lanes;
};

__device__ __forceinline__ uint32_t group_token(const Shape& s, int* lane)
{
  *lane = threadIdx.x & (s.lanes - 1);
  return blockIdx.x * (kThreads / s.lanes) + threadIdx.x / s.lanes;
}

// Rows past the last kept one are zeros: group t clears every tokens-th of
// them from its own on.
template <class U>
__device__ __forceinline__ void clear_tail(const Shape& s, const int64_t* kept, uint32_t t, int lane, int64_t units,
                                           U* rows)
{
  const int64_t slots = (int64_t)s.tokens * s.k;
  for (int64_t r = max(*kept, (int64_t)0) + t; r < slots; r += s.tokens)
    for (int64_t c = lane; c < units; c += s.lanes)
      rows[r * units + c] = U{};
}

// U units of a token's row at a time, from the lane's first on.
template <int U, class T>
__device__ __forceinline__ void copy_units(const T* x, const Shape& s, const int32_t* at, int lane, T* rows)
{
  const uint32_t slots = s.tokens * (uint32_t)s.k;
  for (int64_t c0 = lane; c0 < s.width; c0 += U * s.lanes) {
    T v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * s.lanes < s.width)
        v[u] = x[c0 + u * s.lanes];
    for (int j = 0; j < s.k; ++j) {
      const int32_t r = row_at(at + j, slots);
      if (r >= 0) {
        T* to = rows + (int64_t)r * s.width;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c0 + u * s.lanes < s.width)
            to[c0 + u * s.lanes] = v[u];
      }
    }
  }
}

// Elements are moved as they are: T is an unsigned integer of their size or
// of several of them. Bound by the k rows written for each one read.
template <class T>
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const T* x, int64_t stride, Shape s, const int32_t* row_of_slot, const int64_t* kept, T* rows)
{
  wait_for_previous();
  allow_next();
  int lane;
  const uint32_t t = group_token(s, &lane);
  if (t >= s.tokens)
    return;
  x += (int64_t)t * stride;
  const int32_t* at = row_of_slot + (int64_t)t * s.k;
  if (s.width <= s.lanes)
    copy_units<1>(x, s, at, lane, rows);
  else
    copy_units<4>(x, s, at, lane, rows);
  clear_tail(s, kept, t, lane, s.width, rows);
}

// A group of threads per token, eight rows in flight in registers: for few
// tokens, and for rows that cannot be copied asynchronously (N = 1: their
// parts do not start on 16-byte boundaries).
template <class T, int N, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads, 3)
combine_kernel(const T* rows, int64_t stride, Shape s, const int32_t* row_of_slot, const float* weights, T* out)
{
  wait_for_previous();
  allow_next();
  int lane;
  const uint32_t t = group_token(s, &lane);
  if (t >= s.tokens)
    return;
  const int32_t* at = row_of_slot + (int64_t)t * s.k;
  const uint32_t slots = s.tokens * (uint32_t)s.k;
  const float* w = weights + (int64_t)t * s.k;
  constexpr int P = kPart<N>;
  for (int64_t c = part_start<N>(lane); c < s.width; c += (int64_t)s.lanes * P) {
    float acc[P] = {};
    // eight rows in flight; summed in the order of the slots
    for (int j0 = 0; j0 < s.k; j0 += 8) {
      Part<T, N> v[8];
      int32_t r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = j0 + j < s.k ? row_at(at + j0 + j, slots) : -1;
        if (r[j] >= 0)
          v[j] = load_part<T, N>(rows + r[j] * stride + c, s.lanes, s.width - c);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (r[j] < 0)
          continue;
        const float wj = WEIGHTED ? w[j0 + j] : 1.0f;
#pragma unroll
        for (int i = 0; i < P; ++i)
          acc[i] = fmaf(wj, v[j].f32(i), acc[i]);
      }
    }
    store_part<T, N>(out + (int64_t)t * s.width + c, acc, s.lanes, s.width - c);
  }
}

// The backward pass for rows that cannot be copied asynchronously: a group of
// threads per token, element by element.
template <class T>
__global__ void __launch_bounds__(kThreads, 3)
combine_backward_kernel(const T* grad, int64_t grad_stride, const T* rows, int64_t stride, Shape s,
                        const int32_t* row_of_slot, const float* weights, const int64_t* kept, T* grad_rows,
                        float* grad_weights)
{
  constexpr int P = kPart<1>;
  __shared__ float part[kThreads / 32][8];
  wait_for_previous();
  allow_next();
  int lane;
  const uint32_t t = group_token(s, &lane);
  // whole blocks go on where a group spans several warps; otherwise the
  // groups of a warp that have no token only take part in its reductions
  const bool some = t < s.tokens;
  const int32_t* at = row_of_slot + (int64_t)t * s.k;
  const uint32_t slots = s.tokens * (uint32_t)s.k;
  const float* w = weights + (int64_t)t * s.k;
  for (int j0 = 0; j0 < s.k; j0 += 8) {
    int32_t r[8];
    float wj[8], dot[8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[j] = some && j0 + j < s.k ? row_at(at + j0 + j, slots) : -1;
      wj[j] = r[j] >= 0 ? w[j0 + j] : 0.0f;
    }
    if (some)
      for (int64_t c = part_start<1>(lane); c < s.width; c += (int64_t)s.lanes * P) {
        const int64_t left = s.width - c;
        const Part<T, 1> g = load_part<T, 1>(grad + (int64_t)t * grad_stride + c, s.lanes, left);
        Part<T, 1> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r[j] >= 0)
            v[j] = load_part<T, 1>(rows + r[j] * stride + c, s.lanes, left);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (r[j] < 0)
            continue;
          float y[P];
#pragma unroll
          for (int i = 0; i < P; ++i) {
            dot[j] = fmaf(v[j].f32(i), g.f32(i), dot[j]); // zeros past the row's end
            y[i] = wj[j] * g.f32(i);
          }
          store_part<T, 1>(grad_rows + r[j] * s.width + c, y, s.lanes, left);
        }
      }
    // the lanes' parts of each product, always added in the same order
#pragma unroll
    for (int j = 0; j < 8; ++j)
      for (int o = min(s.lanes, 32) / 2; o > 0; o >>= 1)
        dot[j] += __shfl_xor_sync(kAll, dot[j], o);
    if (s.lanes > 32) {
      const int warp = threadIdx.x >> 5;
      __syncthreads(); // part may still be read
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          part[warp][j] = dot[j];
      __syncthreads();
      if (lane < 8) {
        dot[0] = 0;
        for (int v = 0; v < s.lanes / 32; ++v)
          dot[0] += part[warp + v][lane];
      }
      if (some && lane < 8 && j0 + lane < s.k)
        grad_weights[(int64_t)t * s.k + j0 + lane] = dot[0];
    } else if (some && lane == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < s.k)
          grad_weights[(int64_t)t * s.k + j0 + j] = dot[j];
    }
  }
  if (some)
    clear_tail(s, kept, t, lane, s.width, grad_rows);
}

// Many tokens: a group of threads takes a run of them and copies the next
// kAhead rows into shared memory meanwhile, across tokens. Four blocks of 48
// KB an SM keep 192 KB under way; eight rows a thread in registers, 96 KB
// while a block lasts and nothing while the next one starts (58 us and 102
// for the sum and its backward above, 392 for the larger sum).
constexpr int kAhead = kRingBytes / (kThreads * 16);
constexpr int kAheadBack = kAhead - 1; // leaves room for the products' parts

struct Run {
  Shape s;
  uint32_t groups;
  uint32_t at, end; // tokens of this thread's group, as set by start()
  int lane;
  __device__ __forceinline__ uint32_t start()
  {
    lane = threadIdx.x & (s.lanes - 1);
    const uint32_t g = blockIdx.x * (kThreads / s.lanes) + threadIdx.x / s.lanes;
    at = g < groups ? (uint32_t)((uint64_t)s.tokens * g / groups) : 0;
    end = g < groups ? (uint32_t)((uint64_t)s.tokens * (g + 1) / groups) : 0;
    return g;
  }
};

template <class T, int N, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads, 4)
combine_run_kernel(const T* rows, int64_t stride, Run run, const int32_t* row_of_slot, const float* weights, T* out)
{
  extern __shared__ uint4 ring[];
  wait_for_previous();
  allow_next();
  run.start();
  const int64_t c = ((int64_t)blockIdx.y * run.s.lanes + run.lane) * N;
  if (c >= run.s.width || run.at == run.end)
    return;
  rows += c;
  out += c;
  const int k = run.s.k;
  const uint32_t slots = run.s.tokens * (uint32_t)k, last = run.end * (uint32_t)k;
  uint32_t ahead = run.at * (uint32_t)k; // the next slot to copy
  auto copy = [&](int at) {
    if (ahead < last) {
      const int32_t r = row_at(row_of_slot + ahead, slots);
      if (r >= 0)
        copy_async<16>(&ring[at * kThreads + threadIdx.x], rows + r * stride);
      ++ahead;
    }
    commit_copies();
  };
  for (int u = 0; u < kAhead; ++u)
    copy(u);
  float acc[N] = {};
  uint32_t t = run.at;
  int at = 0, j = 0;
  for (uint32_t i = run.at * (uint32_t)k; i < last; ++i) {
    const int32_t r = row_at(row_of_slot + i, slots);
    const float w = WEIGHTED ? weights[i] : 1.0f;
    wait_for_copies<kAhead - 1>();
    if (r >= 0) {
      const Vec<T, N> v = load<T, N>(reinterpret_cast<const T*>(&ring[at * kThreads + threadIdx.x]));
#pragma unroll
      for (int e = 0; e < N; ++e)
        acc[e] = fmaf(w, v.f32(e), acc[e]);
    }
    copy(at);
    at = at + 1 == kAhead ? 0 : at + 1;
    if (++j == k) {
      store_f32<T, N>(out + (int64_t)t * run.s.width, acc);
#pragma unroll
      for (int e = 0; e < N; ++e)
        acc[e] = 0;
      ++t;
      j = 0;
    }
  }
}

// Sums over a warp of eight values of each lane, in nine exchanges instead of
// forty: at each of the first three a lane passes on half of the values that
// it still has. The result in lane l is the sum of value l / 4.
__device__ __forceinline__ float warp_sum8(float (&v)[8])
{
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 4, o = 16; n > 0; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float pass = upper ? v[i] : v[i + n];
      v[i] = (upper ? v[i + n] : v[i]) + __shfl_xor_sync(kAll, pass, o);
    }
  }
  v[0] += __shfl_xor_sync(kAll, v[0], 2);
  return v[0] + __shfl_xor_sync(kAll, v[0], 1);
}

template <class T, int N>
__global__ void __launch_bounds__(kThreads, 4)
combine_backward_run_kernel(const T* grad, int64_t grad_stride, const T* rows, int64_t stride, Run run,
                            const int32_t* row_of_slot, const float* weights, const int64_t* kept, T* grad_rows,
                            float* grad_weights)
{
  extern __shared__ uint4 ring[];
  __shared__ float part[2][kThreads / 32][8];
  wait_for_previous();
  allow_next();
  const uint32_t group = run.start();
  const int lanes = run.s.lanes, lane = run.lane, k = run.s.k;
  const int64_t width = run.s.width, step = (int64_t)lanes * N, c0 = (int64_t)lane * N;
  const uint32_t slots = run.s.tokens * (uint32_t)k;
  // Copies, for each token, eight of its slots at a time and each of the
  // thread's columns: the gradient's part, then the rows'. The order is that
  // of the loops below.
  struct {
    uint32_t t;
    int j0, u; // u 0: the gradient, else slot j0 + u - 1
    int64_t c;
  } ahead = {run.at, 0, 0, c0};
  auto copy = [&](int at) {
    if (ahead.t < run.end) {
      const T* from = nullptr;
      if (ahead.u == 0) {
        from = grad + (int64_t)ahead.t * grad_stride;
      } else {
        const int32_t r = row_at(row_of_slot + (ahead.t * (uint32_t)k + ahead.j0 + ahead.u - 1), slots);
        if (r >= 0)
          from = rows + r * stride;
      }
      if (from && ahead.c < width)
        copy_async<16>(&ring[at * kThreads + threadIdx.x], from + ahead.c);
      if (++ahead.u > min(8, k - ahead.j0)) {
        ahead.u = 0;
        ahead.c += step;
        if (ahead.c - c0 >= width) {
          ahead.c = c0;
          ahead.j0 += 8;
          if (ahead.j0 >= k) {
            ahead.j0 = 0;
            ++ahead.t;
          }
        }
      }
    }
    commit_copies();
  };
  for (int u = 0; u < kAheadBack; ++u)
    copy(u);
  int at = 0, turn = 0;
  auto take = [&]() { // the next copied part; its place is copied to again
    wait_for_copies<kAheadBack - 1>();
    const Vec<T, N> v = load<T, N>(reinterpret_cast<const T*>(&ring[at * kThreads + threadIdx.x]));
    copy(at);
    at = at + 1 == kAheadBack ? 0 : at + 1;
    return v;
  };
  for (uint32_t t = run.at; t < run.end; ++t) {
    for (int j0 = 0; j0 < k; j0 += 8) {
      const uint32_t i0 = t * (uint32_t)k + j0;
      float dot[8] = {};
      for (int64_t c = c0; c - c0 < width; c += step) {
        const Vec<T, N> g = take();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j0 + j >= k)
            break;
          const Vec<T, N> v = take();
          const int32_t r = row_at(row_of_slot + i0 + j, slots);
          if (r < 0 || c >= width)
            continue;
          const float w = weights[i0 + j];
          float y[N];
#pragma unroll
          for (int e = 0; e < N; ++e) {
            dot[j] = fmaf(v.f32(e), g.f32(e), dot[j]);
            y[e] = w * g.f32(e);
          }
          store_f32<T, N>(grad_rows + r * width + c, y);
        }
      }
      // the lanes' parts of each product, always added in the same order
      if (lanes < 32) {
        const unsigned mask = ((1u << lanes) - 1) << ((threadIdx.x & 31) - lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          for (int o = lanes / 2; o > 0; o >>= 1)
            dot[j] += __shfl_xor_sync(mask, dot[j], o);
          if (lane == 0 && j0 + j < k)
            grad_weights[i0 + j] = dot[j];
        }
        continue;
      }
      const float sum = warp_sum8(dot);
      const int j = (threadIdx.x & 31) / 4;
      if (lanes == 32) {
        if (lane % 4 == 0 && j0 + j < k)
          grad_weights[i0 + j] = sum;
        continue;
      }
      const int warp = threadIdx.x >> 5;
      if (lane % 4 == 0)
        part[turn][warp][j] = sum;
      // the group's warps only; the two turns' memory makes one barrier do
      asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / lanes), "r"(lanes) : "memory");
      if (lane < 8 && j0 + lane < k) {
        float all = 0;
        for (int v = 0; v < lanes / 32; ++v)
          all += part[turn][warp + v][lane];
        grad_weights[i0 + lane] = all;
      }
      turn ^= 1;
    }
  }
  if (group < run.groups)
    for (int64_t r = max(*kept, (int64_t)0) + group; r < slots; r += run.groups)
      for (int64_t c = c0; c < width; c += step)
        store<T, N>(grad_rows + r * width + c, Vec<T, N>{});
}

// Groups resident at four blocks an SM where a token's columns take `tiles`
// groups.
int64_t resident(const Shape& s, int64_t tiles, int sms)
{
  return std::max<int64_t>(1, (int64_t)sms * 4 * kThreads / (s.lanes * tiles));
}
// Whole waves of resident groups, of as many as leave runs of eight tokens or
// more. 8192 tokens of 2048 in bf16, k = 8, in runs of 1, 3, 8, 13 (one
// wave): 62, 53, 53, 50 us; 32768 of 4096 in runs of 7, 27, 108: 353, 364, 369.
Run run_of(const Shape& s, int64_t tiles, int sms)
{
  const int64_t groups = resident(s, tiles, sms);
  return {s, (uint32_t)std::min<int64_t>(s.tokens, groups * std::max<int64_t>(1, s.tokens / (8 * groups))), 0, 0, 0};
}
constexpr int64_t kMaxTilesOfGrid = 65535; // they are grid.y
dim3 grid_of(const Run& run, int64_t tiles)
{
  const uint32_t per_block = (uint32_t)(kThreads / run.s.lanes);
  return dim3((run.groups + per_block - 1) / per_block, (unsigned)tiles);
}

dim3 grid_of(const Shape& s)
{
  const uint32_t per_block = (uint32_t)(kThreads / s.lanes);
  return dim3((s.tokens + per_block - 1) / per_block);
}

int check(int64_t tokens, int32_t k, int64_t width)
{
  if (tokens < 0 || k < 1 || width < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (tokens > 2147483647LL / k)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  return SEGTOPK_SUCCESS;
}

} // namespace
} // namespace segtopk

using namespace segtopk;

extern "C" int segtopk_dispatch(const void* x, int32_t element_bytes, int64_t tokens, int32_t k, int64_t width,
                                int64_t x_stride, const int32_t* row_of_slot, const int64_t* kept, void* rows,
                                void* stream)
{
  record_launch_count(0);
  int rc = check(tokens, k, width);
  if (rc != SEGTOPK_SUCCESS)
    return rc;
  if ((element_bytes != 1 && element_bytes != 2 && element_bytes != 4 && element_bytes != 8) ||
      x_stride < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (tokens == 0 || width == 0)
    return SEGTOPK_SUCCESS;
  if (!x || !row_of_slot || !kept || !rows)
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (!aligned(x, element_bytes) || !aligned(rows, element_bytes) || !aligned(row_of_slot, 4) || !aligned(kept, 8))
    return SEGTOPK_ERROR_MISALIGNED;
  int sms;
  if ((rc = check_device(&sms)) != SEGTOPK_SUCCESS)
    return rc;
  // the widest unit that every row starts on and consists of
  const uint64_t row = (uint64_t)width * element_bytes;
  const uint64_t step = tokens > 1 ? (uint64_t)x_stride * element_bytes : 0;
  const uint64_t bits = (uint64_t)(uintptr_t)x | (uint64_t)(uintptr_t)rows | row | step;
  auto move = [&](auto unit) {
    using T = decltype(unit);
    const int64_t units = (int64_t)(row / sizeof(T));
    // a thread for every 16 bytes, so that few tokens are soon done (1237
    // rows of 4000 bytes, k = 6: 5.4 us, with four units a thread 6.4); of
    // smaller units each takes four
    const Shape s = {(uint32_t)tokens, k, units, lanes_for(sizeof(T) == 16 ? units : (units + 3) / 4, kThreads)};
    return finish(launch(dispatch_kernel<T>, grid_of(s), kThreads, 0, (cudaStream_t)stream, (const T*)x,
                         (int64_t)(step / sizeof(T)), s, row_of_slot, kept, (T*)rows), 1);
  };
  if (bits % 16 == 0)
    return move(uint4{});
  if (bits % 8 == 0)
    return move(uint64_t{});
  if (bits % 4 == 0)
    return move(uint32_t{});
  return bits % 2 == 0 ? move(uint16_t{}) : move(uint8_t{});
}

extern "C" int segtopk_combine(segtopk_dtype dtype, const void* rows, int64_t tokens, int32_t k, int64_t width,
                               int64_t row_stride, const int32_t* row_of_slot, const float* weights, void* out,
                               void* stream)
{
  record_launch_count(0);
  int rc = check(tokens, k, width);
  if (rc != SEGTOPK_SUCCESS)
    return rc;
  if (dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 || row_stride < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  return with_float_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    constexpr int N = 16 / (int)sizeof(T);
    if (tokens == 0 || width == 0)
      return (int)SEGTOPK_SUCCESS;
    if (!rows || !row_of_slot || !out)
      return (int)SEGTOPK_ERROR_INVALID_VALUE;
    if (!aligned(rows, sizeof(T)) || !aligned(out, sizeof(T)) || !aligned(row_of_slot, 4) || !aligned(weights, 4))
      return (int)SEGTOPK_ERROR_MISALIGNED;
    int sms;
    const int bad = check_device(&sms);
    if (bad != SEGTOPK_SUCCESS)
      return bad;
    auto go = [&](auto n) {
      constexpr int V = decltype(n)::value;
      const Shape s = {(uint32_t)tokens, k, width, lanes_for(parts_of(width, V), kThreads)};
      if constexpr (V > 1) {
        const int64_t cols = (int64_t)s.lanes * V, tiles = (width + cols - 1) / cols;
        // runs pay once they are long: 1237 tokens of 1000 in f32, k = 6, take
        // 6.1 us a token per group and 7.1 in runs of two; 8192 of 2048 in
        // bf16 58 and 50. Rows of more tiles than a grid has (67 million
        // columns in f32) go by the other kernel, which loops over columns.
        if (tokens >= 8 * resident(s, tiles, sms) && tiles <= kMaxTilesOfGrid) {
          const Run run = run_of(s, tiles, sms);
          auto kernel = weights ? combine_run_kernel<T, V, true> : combine_run_kernel<T, V, false>;
          return finish(launch(kernel, grid_of(run, tiles), kThreads, kRingBytes, (cudaStream_t)stream, (const T*)rows,
                               row_stride, run, row_of_slot, weights, (T*)out), 1);
        }
      }
      auto kernel = weights ? combine_kernel<T, V, true> : combine_kernel<T, V, false>;
      return finish(launch(kernel, grid_of(s), kThreads, 0, (cudaStream_t)stream, (const T*)rows, row_stride, s,
                           row_of_slot, weights, (T*)out), 1);
    };
    if (rows_fit(rows, row_stride, width, sizeof(T), N) && rows_fit(out, width, width, sizeof(T), N))
      return go(std::integral_constant<int, N>{});
    return go(std::integral_constant<int, 1>{});
  });
}

extern "C" int segtopk_combine_backward(segtopk_dtype dtype, const void* grad_out, int64_t grad_stride,
                                        const void* rows, int64_t row_stride, int64_t tokens, int32_t k,
                                        int64_t width, const int32_t* row_of_slot, const int64_t* kept,
                                        const float* weights, void* grad_rows, float* grad_weights, void* stream)
{
  record_launch_count(0);
  int rc = check(tokens, k, width);
  if (rc != SEGTOPK_SUCCESS)
    return rc;
  if (dtype < SEGTOPK_F16 || dtype > SEGTOPK_I32 || row_stride < 0 ||
      grad_stride < 0)
    return SEGTOPK_ERROR_INVALID_VALUE;
  return with_float_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    constexpr int N = 16 / (int)sizeof(T);
    if (tokens == 0)
      return (int)SEGTOPK_SUCCESS;
    if (!row_of_slot || !kept || !weights || !grad_weights || (width > 0 && (!grad_out || !rows || !grad_rows)))
      return (int)SEGTOPK_ERROR_INVALID_VALUE;
    if (!aligned(grad_out, sizeof(T)) || !aligned(rows, sizeof(T)) || !aligned(grad_rows, sizeof(T)) ||
        !aligned(row_of_slot, 4) || !aligned(kept, 8) || !aligned(weights, 4) || !aligned(grad_weights, 4))
      return (int)SEGTOPK_ERROR_MISALIGNED;
    int sms;
    const int bad = check_device(&sms);
    if (bad != SEGTOPK_SUCCESS)
      return bad;
    auto go = [&](auto n) {
      constexpr int V = decltype(n)::value;
      const Shape s = {(uint32_t)tokens, k, width, lanes_for(parts_of(width, V), kThreads)};
      if constexpr (V > 1) {
        const Run run = run_of(s, 1, sms);
        return finish(launch(combine_backward_run_kernel<T, V>, grid_of(run, 1), kThreads, kAheadBack * kThreads * 16,
                             (cudaStream_t)stream, (const T*)grad_out, grad_stride, (const T*)rows, row_stride, run,
                             row_of_slot, weights, kept, (T*)grad_rows, grad_weights), 1);
      }
      return finish(launch(combine_backward_kernel<T>, grid_of(s), kThreads, 0, (cudaStream_t)stream,
                           (const T*)grad_out, grad_stride, (const T*)rows, row_stride, s, row_of_slot, weights, kept,
                           (T*)grad_rows, grad_weights), 1);
    };
    if (rows_fit(grad_out, grad_stride, width, sizeof(T), N) && rows_fit(rows, row_stride, width, sizeof(T), N) &&
        rows_fit(grad_rows, width, width, sizeof(T), N))
      return go(std::integral_constant<int, N>{});
    return go(std::integral_constant<int, 1>{});
  });
}
