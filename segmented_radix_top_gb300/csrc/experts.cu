// Rows moved to expert order and back (segtopk_dispatch, segtopk_combine and
// segtopk_combine_backward in include/segtopk.h).
//
//   dispatch          rows[r(t, j)] = x[t]
//   combine           out[t] = sum_j w_tj rows[r(t, j)]
//   combine backward  grad_rows[r(t, j)] = w_tj g[t],  grad_w_tj = <rows[r(t, j)], g[t]>
//
// r(t, j) is the row of token t's j-th slot, or none. Every kernel goes by
// token, so a token's row is read or written once and only the k sorted rows
// are scattered; all are bound by memory bandwidth.
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

// Elements are moved as they are: T is an unsigned integer of their size or
// of several of them.
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
  const int32_t* at = row_of_slot + (int64_t)t * s.k;
  const uint32_t slots = s.tokens * (uint32_t)s.k;
  for (int64_t c = lane; c < s.width; c += s.lanes) {
    const T v = x[(int64_t)t * stride + c];
    for (int j = 0; j < s.k; ++j) {
      const int32_t r = row_at(at + j, slots);
      if (r >= 0)
        rows[(int64_t)r * s.width + c] = v;
    }
  }
  clear_tail(s, kept, t, lane, s.width, rows);
}

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
  for (int64_t c = (int64_t)lane * N; c < s.width; c += (int64_t)s.lanes * N) {
    float acc[N] = {};
    // eight rows in flight; summed in the order of the slots
    for (int j0 = 0; j0 < s.k; j0 += 8) {
      Vec<T, N> v[8];
      int32_t r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = j0 + j < s.k ? row_at(at + j0 + j, slots) : -1;
        if (r[j] >= 0)
          v[j] = load<T, N>(rows + r[j] * stride + c);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (r[j] < 0)
          continue;
        const float wj = WEIGHTED ? *(w + j0 + j) : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
          acc[i] = fmaf(wj, v[j].f32(i), acc[i]);
      }
    }
    store_f32<T, N>(out + (int64_t)t * s.width + c, acc);
  }
}

template <class T, int N>
__global__ void __launch_bounds__(kThreads, 3)
combine_backward_kernel(const T* grad, int64_t grad_stride, const T* rows, int64_t stride, Shape s,
                        const int32_t* row_of_slot, const float* weights, const int64_t* kept, T* grad_rows,
                        float* grad_weights)
{
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
      wj[j] = r[j] >= 0 ? *(w + j0 + j) : 0.0f;
    }
    if (some)
      for (int64_t c = (int64_t)lane * N; c < s.width; c += (int64_t)s.lanes * N) {
        float g[N];
        const Vec<T, N> got = load<T, N>(grad + (int64_t)t * grad_stride + c);
#pragma unroll
        for (int i = 0; i < N; ++i)
          g[i] = got.f32(i);
        Vec<T, N> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r[j] >= 0)
            v[j] = load<T, N>(rows + r[j] * stride + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (r[j] < 0)
            continue;
          float y[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot[j] = fmaf(v[j].f32(i), g[i], dot[j]);
            y[i] = wj[j] * g[i];
          }
          store_f32<T, N>(grad_rows + r[j] * s.width + c, y);
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
    clear_tail(s, kept, t, lane, s.width / N, reinterpret_cast<Vec<T, N>*>(grad_rows));
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
    const Shape s = {(uint32_t)tokens, k, (int64_t)(row / sizeof(T)), lanes_for((int64_t)(row / sizeof(T)), kThreads)};
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
      const Shape s = {(uint32_t)tokens, k, width, lanes_for(width / V, kThreads)};
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
      const Shape s = {(uint32_t)tokens, k, width, lanes_for(width / V, kThreads)};
      return finish(launch(combine_backward_kernel<T, V>, grid_of(s), kThreads, 0, (cudaStream_t)stream,
                           (const T*)grad_out, grad_stride, (const T*)rows, row_stride, s, row_of_slot, weights, kept,
                           (T*)grad_rows, grad_weights), 1);
    };
    if (rows_fit(grad_out, grad_stride, width, sizeof(T), N) && rows_fit(rows, row_stride, width, sizeof(T), N) &&
        rows_fit(grad_rows, width, width, sizeof(T), N))
      return go(std::integral_constant<int, N>{});
    return go(std::integral_constant<int, 1>{});
  });
}
